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
// their rows are tokens, and then columns of values.  The work is cut among the warps of the
// whole GPU: each walks a share of its own, in steps of 32 tokens, with a running maximum and
// sum and 8 NT x D sums, and leaves what it has of a unit as a partial.  (Cut among CTAs, whose
// warps took turns and met at the end of every unit, 128 caches of up to 16384 tokens took
// 344 us.)  A warp copies its steps itself, by cp.async into slots of its own,
// the next ones while it works on one, on into the next piece.  (Bulk copies by one warp
// took 80 clocks each to issue, 1900 to 2600 per 128 tokens: more than all the rest.)
// Per 16 tokens:
//     S^T = K Q^T        K in bf16 (exactly), contracted over D in an order of its own:
//                        lane j of four has columns j D/4 .. of a token, 16 adjacent bytes
//     P = 2^(S scale log2(e) - m), rounded to fp16; m moves when a weight would pass 2^15, to 7
//                        below the maximum, so that a weight loses 2^-11 of it, or 2^-32 of the largest
//                        where it is below 2^-21 of that (bf16 would lose 2^-8; the sum is of the
//                        weights before they are rounded)
//     O^T += V^T P^T     V in fp16 as eighths (exactly); lane r of eight has the D / 8 columns
//                        from r D/8 on, two of them rows r and r + 8 of each product
// The 16 rows of a product are tokens in the order 0 4 1 5 2 6 3 7, 8 12 .., so that the tokens
// whose values four lanes read are adjacent, and both reads are free of bank conflicts.  P^T
// comes from S^T's fragments by an 8 x 8 transposition in the warp.
//
// 128 caches of up to 16384 tokens, a row of 8 query heads on each of 8 (911 MB): 247 us, 3.7 TB/s, 0.54 of a plain copy's rate;
// 64 caches of up to 8192, up to 9 rows of 4 query heads: 128 us.  56 % of the issue slots are used (twelve warps an SM, three for a
// scheduler; counters of half of the tokens), 44 % of the integer pipe, 26 % of the fp16 one, 17 % of the matrix pipe: no
// pipe is full.  A warp's own chain bounds it -- keys, S, vote, weights, transposition, values -- and three warps do not
// fill its waits.  Most of its instructions unpack: per two elements a mask with an exponent, 3/4 of a shift for
// keys, 1/4 and as many byte permutations for values, and one (keys) or two (values) fp16 operations,
// all of half the rate of fp32; 32 NT matrix products of 8 clocks.  MmaShape<128, 2, true> spills 12 bytes a thread at
// 168 registers.  Head sizes between 64 and 128 run as 128 with columns of zeros: D = 80 and 96 take as long as 128 does.
#include <new>

#include "attn_tc_kernel.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kStepLog2 = 5, kStep = 1 << kStepLog2;  // tokens of a step
constexpr int kMmaTileLog2 = 6;                       // of a tile, the least that a warp has of a unit
constexpr float kLift = 7.f;  // the reference stands below the maximum, as in attn_tc_kernel.cuh
constexpr int kMmaMostShare = kMostShare >> 4;  // places of a warp's share: its SM's twelve are minutes of work
constexpr int kMmaUnitCost = 2;  // tiles: a unit's start and end (1 and 2 measured alike, 4 and 8 by 3 to 6 % worse)

// A warp's place in its share: the piece that it works on and the next one, and the walk
// (in shared memory: they are looked at between pieces).
struct Pieces {
    Piece x[2];
    Walk<Params> walk;
};

// DP: D padded, NT: lines / 8, FULL: D is DP
template <int DP_, int NT_, bool FULL_>
struct MmaShape {
    static constexpr int DP = DP_, NT = NT_;
    static constexpr bool FULL = FULL_;
    static constexpr int NW = 12, kThreads = 32 * NW;   // 168 registers a thread
    static constexpr int kSlot = kStep * DP / 16 * 18;  // codes of keys, of values, scales of keys, of values
    static constexpr int kQ = NT == 1 ? 0 : NT * DP / 16 * 256;  // uint2 [DP / 16][32][NT]; with 8 lines they stay in registers
    static constexpr int kPieces = (int)(sizeof(Pieces) + 15) / 16 * 16;
    static constexpr int kDepth = NT == 1 ? 4 : 3;      // slots, a step each
    static constexpr int kWarp = kDepth * kSlot + kQ + kPieces;
    static constexpr int kSmem = NW * kWarp;
    static_assert(kSlot % 16 == 0, "places");
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
// steps of a piece: the first one, and the one after its last
__device__ __forceinline__ int first_step(const Piece &x) { return x.t0 << (kMmaTileLog2 - kStepLog2); }
__device__ __forceinline__ int last_step(const Piece &x) {
    return min(x.t1 << (kMmaTileLog2 - kStepLog2), (int)(((unsigned)x.tokens + kStep - 1) >> kStepLog2));
}

// ---------------------------------------------------------------- a warp's copies
// The next step to copy: step t of the warp's piece `piece` (counted over its pieces, the one
// after the piece worked on at most), its first token and the pages of its four groups of
// eight tokens (lane % 4), fetched a step ahead.
struct Copies {
    int piece, t, t1;  // t >= t1: none is left in the piece
    int tok0, last;    // first token of the step; the unit's last one
    int page, off;     // of this lane's group: page, token in it
    int h;             // key-value head
    uint32_t issued, used;

    __device__ __forceinline__ bool any() const { return t < t1; }
};
__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// ---------------------------------------------------------------- the kernel
// fragment of the first product of a unit's queries: columns d .. d + 3 of line `line`, zero beyond the unit and D
__device__ __forceinline__ uint2 query_of(const Params &p, const Piece &x, int line, int d) {
    const dspark_tree_attention_args &a = p.a;
    const int h = x.head / p.subs, sub = x.head - h * p.subs, jj = line / p.heads, g = line - jj * p.heads;
    if (jj >= x.n || sub * p.heads + g >= p.G || d >= a.D) return make_uint2(0u, 0u);
    return *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + (long long)(x.row0 + x.first + jj) * a.q_row +
                                            (h * p.G + sub * p.heads + g) * a.q_head + d);
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention4_mma(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int DP = C::DP, NT = C::NT, KS = DP / 16, MT = DP / 16, ND = DP / 8;  // steps of the first product, rows / 16 of the second, columns of a lane
    const dspark_tree_attention_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    after_predecessor();
    const int D = C::FULL ? DP : a.D, code_row = D / 2, scale_row = D / 16;
    // tokens that are adjacent in a page and in a step: copied from one address
    const int run = min(kStep, a.page & -a.page);
    const float scale = fmaxf(p.scale_log2, 1e-37f);  // 0 would make -inf x 0 of what is not seen
    const int token_r = (r >> 1) + 4 * (r & 1);  // token of a product's row r; of row r + 8 eight on
    unsigned char *slots = smem + warp * C::kWarp;
    uint2 *q = reinterpret_cast<uint2 *>(slots + C::kDepth * C::kSlot);
    Pieces &mine = *reinterpret_cast<Pieces *>(slots + C::kDepth * C::kSlot + C::kQ);
    const int cta = blockIdx.x * C::NW + warp;  // of as many shares as there are warps
    {
        const Share share = share_of(p, cta, gridDim.x * C::NW, kMmaMostShare);
        if (lane == 0) {
            p.join[cta].pieces = 0;
            new (&mine.walk) Walk<Params>(p, share);
        }
    }
    // takes the next piece of the walk into its place (n: counted over the warp's pieces); r < 0: none is left
    auto take = [&](int n) {
        if (lane == 0) {
            Piece &y = mine.x[n & 1];
            if (!mine.walk.next(y)) y.r = -1;
            else if (y.t0 == 0 && y.t1 < y.tiles) p.join[cta] = mine.walk.join_of(y);
        }
        __syncwarp();
    };
    int now = 0;  // the piece worked on
    Copies cp{-1, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    // to the next step, in the piece worked on or the one after it, and its pages
    auto seek = [&]() {
        if (!cp.any()) {
            if (cp.piece > now) return;
            const Piece &y = mine.x[++cp.piece & 1];
            if (y.r < 0) return;
            cp.t = first_step(y);
            cp.t1 = last_step(y);
            cp.last = y.tokens - 1;
            cp.h = p.subs == 1 ? y.head : y.head / p.subs;
        }
        cp.tok0 = cp.t << kStepLog2;
        const int tok = min(cp.tok0 + 8 * j, cp.last & -run), in_table = p.page.of(tok);
        cp.off = tok - in_table * a.page;
        cp.page = a.table[(size_t)mine.x[cp.piece & 1].r * a.max_pages + in_table];
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
        // Eight tokens' codes are adjacent, 4 D bytes, and so are their scales, D / 2.  (Groups beyond the unit's last token
        // get more of its page, or that page's run again; what stands there is not looked at.)
        long long from = 0;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if ((8 * g & (run - 1)) == 0) from = __shfl_sync(0xffffffffu, at + (long long)cp.off * code_row, g) + 16 * lane;
            else from += 8 * code_row;
            if ((C::FULL && DP == 128) || 4 * lane < D) {
                unsigned char *dst = to + 8 * g * code_row + 16 * lane;
                cp_async16(dst, kc + from);
                cp_async16(dst + kStep * code_row, vc + from);
            }
        }
        const int g = lane >> 3, e = lane & 7, first = g & -(run >> 3);  // the group whose address stands for the run
        from = __shfl_sync(0xffffffffu, at + codes + (long long)cp.off * scale_row, first) + 8 * (g - first) * scale_row + 8 * e;
        if ((C::FULL && DP == 128) || 16 * e < D) {
            unsigned char *dst = to + 2 * kStep * code_row + 8 * g * scale_row + 8 * e;
            cp_async8(dst, kc + from);
            cp_async8(dst + kStep * scale_row, vc + from);
        }
        tc::cp_async_commit();
        ++cp.issued;
        ++cp.t;
        seek();
    };
    take(0);
    if (mine.x[0].r < 0) return;
    take(1);
    seek();
    for (;;) {
        const Piece x = mine.x[now & 1];
#pragma unroll 1
        while (cp.any() && cp.issued - cp.used < (uint32_t)C::kDepth) copy();
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
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const uint2 v = query_of(p, x, 8 * i + r, j * (DP / 4) + 4 * k);
                if (NT == 1) q_held[NT == 1 ? k : 0] = v;
                else q[(k * 32 + lane) * NT + i] = v;  // (each lane reads what it wrote)
            }
#pragma unroll 1
        for (int s = first_step(x); s < last_step(x); ++s) {
            int tok0 = s << kStepLog2;
            // copies of this step: the oldest; all but it may be under way where the slots are full
            if (cp.issued - cp.used == (uint32_t)C::kDepth) tc::cp_async_wait<C::kDepth - 1>();
            else tc::cp_async_wait<0>();
            __syncwarp();
            const unsigned char *kcode = slots + (cp.used % C::kDepth) * C::kSlot, *vcode = kcode + kStep * code_row,
                                *kscale = vcode + kStep * code_row, *vscale = kscale + kStep * scale_row;
            const bool tail = tok0 + kStep > x.len + base_rel;
            // 16 tokens at a time (in a loop that is not unrolled 5 % slower, all 32 tokens in one go 4 %)
#pragma unroll
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
                                if (C::FULL || j * (DP / 4) + 16 * g < D) w = *reinterpret_cast<const uint2 *>(at + 8 * g);
                                kw[u][2 * g] = w.x, kw[u][2 * g + 1] = w.y;
                            }
                        }
#pragma unroll
                        for (int g = 0; g < KS / 4; ++g) {
                            const bool in = C::FULL || j * (DP / 4) + 16 * g < D;
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
                                const uint4 two = *reinterpret_cast<const uint4 *>(q + (k * 32 + lane) * NT + i);
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
                        const bool in = C::FULL || r * ND < D;
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
                        if (rel < base_rel || tok0 + i >= x.tokens || r * ND >= D) continue;
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

        // ---------------------------------------------------- the piece's end
        {
            const int h = x.head / p.subs, sub = x.head - h * p.subs;
            const bool whole = x.slot < 0;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float2 sum = l[i];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    sum.x += __shfl_xor_sync(0xffffffffu, sum.x, d);
                    sum.y += __shfl_xor_sync(0xffffffffu, sum.y, d);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int line = 8 * i + 2 * j + u, jj = line / p.heads, g = line - jj * p.heads;
                    if (jj >= x.n || sub * p.heads + g >= p.G) continue;
                    const float M = u ? m[i].y : m[i].x, L = u ? sum.y : sum.x;
                    const float f = (whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f) * 8.f;  // (values were multiplied as eighths)
                    const size_t at = (size_t)(x.row0 + x.first + jj) * a.Hq + h * p.G + sub * p.heads + g, to = (size_t)(whole ? 0 : x.slot) * p.lines + line;
                    if (C::FULL || r * ND < D) {
                        if (whole) {
                            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + at * D + r * ND;
#pragma unroll
                            for (int t = 0; t < ND / 2; t += 4)
                                *reinterpret_cast<uint4 *>(out + 2 * t) =
                                    make_uint4(pack(O[i][t][u] * f, O[i][t][2 + u] * f), pack(O[i][t + 1][u] * f, O[i][t + 1][2 + u] * f),
                                               pack(O[i][t + 2][u] * f, O[i][t + 2][2 + u] * f), pack(O[i][t + 3][u] * f, O[i][t + 3][2 + u] * f));
                        } else {
                            float *out = p.part_o + to * p.stride + r * ND;
#pragma unroll
                            for (int t = 0; t < ND / 2; t += 2)
                                *reinterpret_cast<float4 *>(out + 2 * t) =
                                    make_float4(O[i][t][u] * f, O[i][t][2 + u] * f, O[i][t + 1][u] * f, O[i][t + 1][2 + u] * f);
                        }
                    }
                    if (r == 0) {
                        if (!whole) p.part_ml[to] = make_float2(M, L);
                        else if (a.lse) a.lse[at] = lse_of(M, L);
                    }
                }
            }
        }
        // the next piece, which is known, and the one after it
        ++now;
        if (mine.x[now & 1].r < 0) return;
        __syncwarp();
        take(now + 1);
        if (!cp.any()) seek();
    }
}

template <typename C>
cudaError_t launch_mma_as(const Params &p, int grid, cudaStream_t s) {
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    auto kern = tree_attention4_mma<C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, C::kThreads, C::kSmem, s, p);
}

}  // namespace

// shares: one per warp
int mma4_grid() {
    static_assert(MmaShape<128, 1, true>::NW == MmaShape<128, 2, true>::NW, "as many shares as warps, whatever the shape");
    return sm_count() * MmaShape<128, 1, true>::NW;
}

cudaError_t launch_mma4(Params p, int grid, cudaStream_t s) {
    const dspark_tree_attention_args &a = p.a;
    p.tile_log2 = kMmaTileLog2;
    p.small_rows = p.block_rows;
    p.small_places = p.large_places = div_by(1);
    p.page = div_by(a.page);
    p.ctas = div_by(grid);
    p.unit_cost = kMmaUnitCost;
    const int ctas = sm_count();
    if (p.lines <= 8) {
        if (a.D == 128) return launch_mma_as<MmaShape<128, 1, true>>(p, ctas, s);
        if (a.D == 64) return launch_mma_as<MmaShape<64, 1, true>>(p, ctas, s);
        return a.D > 64 ? launch_mma_as<MmaShape<128, 1, false>>(p, ctas, s) : launch_mma_as<MmaShape<64, 1, false>>(p, ctas, s);
    }
    if (a.D == 128) return launch_mma_as<MmaShape<128, 2, true>>(p, ctas, s);
    if (a.D == 64) return launch_mma_as<MmaShape<64, 2, true>>(p, ctas, s);
    return a.D > 64 ? launch_mma_as<MmaShape<128, 2, false>>(p, ctas, s) : launch_mma_as<MmaShape<64, 2, false>>(p, ctas, s);
}

}  // namespace attn
}  // namespace dspark
