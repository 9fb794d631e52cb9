// attn_f32.cu -- attention of drafted rows over a paged cache in fp32 on the CUDA
// cores (D a multiple of 4 up to 128, the caches 16-byte aligned).
//
// A CTA's eight warps split a tile of 64 tokens, eight tokens each, and walk their
// tokens of all tiles by themselves: own copies (cp.async, three stages), own maximum,
// sum and output of the unit's 16 lines, no barrier before the end of a piece, where
// the eight are added like partials.  Per token and line that is D products for the
// score and D for the output, two in one instruction (f32x2).  Shared-memory reads,
// not products, are what there are most of, so a lane works on as large a square as
// its registers hold: 4 lines x 4 tokens over a quarter of the columns for the scores
// (8 16-byte reads per 64 products), 8 lines x 8 columns for the outputs (6 per 64).
// A tile costs the same however few of the 16 lines are in use.  8 query
// heads on 4 of 64: 16 caches of 8192 tokens, 17 rows, 313 us (the general kernel: 730);
// one of 131072, 1 row, 110 (278); 4 of up to 1500, 5 rows, 12.5 (24).
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "attn_tc.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kLines = 16, kTokens = 8, kStages = 3;
constexpr int kTileLog2 = 6;  // 64 = kWarps * kTokens
constexpr float kSlack = 8.f;  // log2 by which a tile may exceed the reference

// floats of a key or query row in shared memory: 64 bytes of padding turn
// neighbouring rows of the same column to the other half of the banks
__host__ __device__ constexpr int row_floats(int D) { return D + 16; }
__host__ __device__ constexpr int stage_floats(int D) { return kTokens * (row_floats(D) + D); }
__host__ __device__ constexpr int warp_floats(int D) { return kStages * stage_floats(D) + 2 * kTokens * kLines; }
constexpr size_t smem_bytes(int D) {
    return sizeof(float) * ((size_t)kLines * row_floats(D) + (size_t)kWarps * warp_floats(D)) + sizeof(float2) * kWarps * kLines;
}

// kWide: D above 64
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1) tree_attention_f32(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float sh[];
    __shared__ Share shared_share;
    const dspark_tree_attention_args &a = p.a;
    const int D = a.D, QS = row_floats(D);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float *sq = sh;
    float *own = sq + kLines * QS + warp * warp_floats(D), *sp = own + kStages * stage_floats(D);
    float2 *sml = reinterpret_cast<float2 *>(sh + kLines * QS + kWarps * warp_floats(D));  // [warp][line]

    after_predecessor();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        const Share s = share_of(p);
        if (lane == 0) {
            shared_share = s;
            p.join[blockIdx.x].pieces = 0;
        }
    }
    __syncthreads();
    Walk walk(p, shared_share);
    // scores: lines lg + 4 i against tokens tg + 2 e over the 16-byte pieces ds, ds + 4, ..
    const int ds = lane & 3, tg = (lane >> 2) & 1, lg = lane >> 3;
    const int ln = lg + 4 * ds;  // the line whose scores (of tokens tg + 2 e) end up here
    // outputs: lines 8 lh + i, columns 4 cg .. + 3 and 64 + 4 cg .. + 3
    const int cg = lane & 15, lh = lane >> 4;
    const int chunks = D / 4;               // 16-byte pieces of a row
    const bool has0 = 4 * cg < D, has1 = kWide && 64 + 4 * cg < D;
    constexpr int kPairs = kWide ? 4 : 2;
    const int at_once = 32 / chunks, sub = lane / chunks, col = lane - sub * chunks;  // copies: rows at once, lane's row and piece
    const float scale = p.scale_log2;
    Piece x;
    while (walk.next(x)) {
        const int h = p.subs == 1 ? x.head : x.head / p.subs, head0 = h * p.G + (p.subs == 1 ? 0 : x.head % p.subs * p.heads);
        const int heads = min(p.heads, (h + 1) * p.G - head0);
        const int32_t *table = a.table + (size_t)x.r * a.max_pages;
        __syncthreads();  // the last piece's queries and sums are read
        // this warp's tokens of tile t into stage `st`; beyond the unit's tokens zeros
        auto token_of = [&](int t) { return min((t << kTileLog2) + warp * kTokens + (lane & 7), x.tokens - 1); };
        auto page_of = [&](int t) { return table[p.page.of(token_of(t))]; };
        auto load = [&](int t, int st, int pg) {
            const int tok0 = (t << kTileLog2) + warp * kTokens;
            if (pg < 0 || pg >= a.n_pages) {
                set_err(a.err, DSPARK_ERR_RANGE);
                pg = 0;
            }
            const int tok = token_of(t), in_page = tok - p.page.of(tok) * a.page;
            const size_t row = (((size_t)pg * a.H + h) * a.page + in_page) * D;  // of token lane & 7
            float *k = own + st * stage_floats(D), *v = k + kTokens * QS;
#pragma unroll 1
            for (int t0 = 0; t0 < kTokens; t0 += at_once) {
                const int tk = t0 + sub;
                const size_t from = __shfl_sync(0xffffffffu, row, tk & 7) + 4 * col;
                if (sub < at_once && tk < kTokens) {
                    const uint32_t bytes = tok0 + tk < x.tokens ? 16u : 0u;
                    tc::cp_async16_zfill(k + tk * QS + 4 * col, static_cast<const float *>(a.k_cache) + from, bytes);
                    tc::cp_async16_zfill(v + tk * D + 4 * col, static_cast<const float *>(a.v_cache) + from, bytes);
                }
            }
        };

        float2 acc[8][kPairs];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < kPairs; ++e) acc[i][e] = make_float2(0.f, 0.f);
        float m = -INFINITY, sum = 0.f;  // of line ln; the sum: of this lane's tokens
        const int row = x.first + ln / p.heads;
        const bool live = ln / p.heads < x.n;
        const uint32_t *words = a.mask && live ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + row) * a.W) : nullptr;

        // a group is committed for every tile, empty or not, so that the count of those
        // under way says which one has landed
        int st = 0, ahead = 0, pg = page_of(x.t0);
        auto load_next = [&](int t) {
            if (t < x.t1) load(t, ahead, pg);
            tc::cp_async_commit();
            if (t + 1 < x.t1) pg = page_of(t + 1);
            ahead = ahead + 1 == kStages ? 0 : ahead + 1;
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) load_next(x.t0 + i);
        // the queries while the first tiles are on their way
        for (int i = tid; i < kLines * D; i += kThreads) {
            const int l = i / D, d = i - l * D, jj = l / p.heads, gl = l - jj * p.heads;
            float v = 0.f;
            if (jj < x.n && gl < heads)
                v = static_cast<const float *>(a.q)[(x.row0 + x.first + jj) * a.q_row + (head0 + gl) * a.q_head + d];
            sq[l * QS + d] = v;
        }
        __syncthreads();

        for (int t = x.t0; t < x.t1; ++t, st = st + 1 == kStages ? 0 : st + 1) {
            load_next(t + kStages - 1);
            tc::cp_async_wait<kStages - 1>();
            __syncwarp();
            const int tok0 = (t << kTileLog2) + warp * kTokens;
            const float *k = own + st * stage_floats(D), *v = k + kTokens * QS;
            float s[4];
            {
                // even and odd products of a score in the two halves of a pair
                float2 z[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[i][e] = make_float2(0.f, 0.f);
                const float *q0 = sq + lg * QS, *k0 = k + tg * QS;
#pragma unroll 2
                for (int d = 4 * ds; d < D; d += 16) {
                    float4 qa[4], kb[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        qa[i] = *reinterpret_cast<const float4 *>(q0 + 4 * i * QS + d);
                        kb[i] = *reinterpret_cast<const float4 *>(k0 + 2 * i * QS + d);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            z[i][e] = fma2({qa[i].x, qa[i].y}, {kb[e].x, kb[e].y}, z[i][e]);
                            z[i][e] = fma2({qa[i].z, qa[i].w}, {kb[e].z, kb[e].w}, z[i][e]);
                        }
                }
                __syncwarp();
                // the four lanes of a quad add their quarters, each for one of the lines
                float h[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float low = z[i][e].x + z[i][e].y, high = z[i + 2][e].x + z[i + 2][e].y;
                        h[i][e] = (ds & 2 ? high : low) + __shfl_xor_sync(0xffffffffu, ds & 2 ? low : high, 2);
                    }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[e] = (ds & 1 ? h[1][e] : h[0][e]) + __shfl_xor_sync(0xffffffffu, ds & 1 ? h[0][e] : h[1][e], 1);
            }
            const bool tail = tok0 + kTokens > x.len;  // rows of this cycle, or slots beyond the unit's tokens
            bool see[4];
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int rel = tok0 + tg + 2 * e - x.len;
                see[e] = true;
                if (tail)
                    see[e] = live && (rel < 0 || (rel < x.rows && (words ? ((words[rel >> 5] >> (rel & 31)) & 1) != 0
                                                                         : !a.mask && rel <= row)));
                s[e] = see[e] ? s[e] * scale : -INFINITY;
                top = fmaxf(top, s[e]);
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            // the reference moves, and the sums with it, when a tile exceeds it by 2^8
            if (__any_sync(0xffffffffu, top > m + kSlack)) {
                const float to = top > m + kSlack ? top : m;
                const float f = to == -INFINITY ? 1.f : ex2(m - to);
                m = to;
                sum *= f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int l = 8 * lh + i;
                    const float fl = __shfl_sync(0xffffffffu, f, (l >> 2) + 8 * (l & 3));  // a lane that has line l
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) acc[i][e].x *= fl, acc[i][e].y *= fl;
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float w = ex2(s[e] - ref);
                sum += w;
                // what the line does not see is marked, so that its value is left out;
                // twice, as the pair that the products take
                const float mark = see[e] ? w : -1.f;
                *reinterpret_cast<float2 *>(sp + 2 * ((tg + 2 * e) * kLines + ln)) = make_float2(mark, mark);
            }
            __syncwarp();
#pragma unroll 2
            for (int tk = 0; tk < kTokens; ++tk) {
                const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 b0 = has0 ? *reinterpret_cast<const float4 *>(v + tk * D + 4 * cg) : zero;
                const float4 b1 = has1 ? *reinterpret_cast<const float4 *>(v + tk * D + 64 + 4 * cg) : zero;
                const float *w = sp + 2 * (tk * kLines + 8 * lh);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 w2 = *reinterpret_cast<const float4 *>(w + 2 * i);  // lines i, i, i + 1, i + 1
                    const float2 pair[2] = {{w2.x, w2.y}, {w2.z, w2.w}};
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        if (tail && pair[o].x < 0.f) continue;
                        acc[i + o][0] = fma2(pair[o], {b0.x, b0.y}, acc[i + o][0]);
                        acc[i + o][1] = fma2(pair[o], {b0.z, b0.w}, acc[i + o][1]);
                        if (kWide) {
                            acc[i + o][kPairs - 2] = fma2(pair[o], {b1.x, b1.y}, acc[i + o][kPairs - 2]);
                            acc[i + o][kPairs - 1] = fma2(pair[o], {b1.z, b1.w}, acc[i + o][kPairs - 1]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage may be copied into
        }

        // the eight warps' parts of the lines, one after the other in shared memory
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        if (tg == 0) sml[warp * kLines + ln] = make_float2(m, sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float *to = own + (8 * lh + i) * D + 4 * cg;
            if (has0) *reinterpret_cast<float4 *>(to) = make_float4(acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y);
            if (has1)
                *reinterpret_cast<float4 *>(to + 64) =
                    make_float4(acc[i][kPairs - 2].x, acc[i][kPairs - 2].y, acc[i][kPairs - 1].x, acc[i][kPairs - 1].y);
        }
        __syncthreads();
        const float *all = sq + kLines * QS;
        for (int i = tid; i < kLines * chunks; i += kThreads) {
            const int l = i / chunks, d = 4 * (i - l * chunks), jj = l / p.heads, gl = l - jj * p.heads;
            if (jj >= x.n || gl >= heads) continue;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[w * kLines + l].x);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = sml[w * kLines + l];
                const float f = ex2(ml.x - ref);
                const float4 y = *reinterpret_cast<const float4 *>(all + w * warp_floats(D) + l * D + d);
                L = fmaf(f, ml.y, L);
                o.x = fmaf(f, y.x, o.x), o.y = fmaf(f, y.y, o.y), o.z = fmaf(f, y.z, o.z), o.w = fmaf(f, y.w, o.w);
            }
            const size_t orow = (size_t)(x.row0 + x.first + jj) * a.Hq + head0 + gl;
            if (x.slot >= 0) {
                const size_t prow = (size_t)x.slot * p.lines + l;
                *reinterpret_cast<float4 *>(p.part_o + prow * p.stride + d) = o;
                if (d == 0) p.part_ml[prow] = make_float2(M, L);
            } else {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                float *out = static_cast<float *>(a.out) + orow * D + d;
                out[0] = o.x * inv, out[1] = o.y * inv, out[2] = o.z * inv, out[3] = o.w * inv;
                if (a.lse && d == 0) a.lse[orow] = lse_of(M, L);
            }
        }
        if (tid == 0 && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
    }
}

}  // namespace

bool f32_supported(const dspark_tree_attention_args &a) {
    return a.dtype == DSPARK_F32 && a.D % 4 == 0 && a.D <= 128 &&
           ((reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache)) & 15) == 0;
}

// one CTA per SM: two (they fit while D is at most 64) have more partials to join,
// and took 16 us instead of 12 for 4 caches of up to 1500 tokens and 68 instead of
// 64 for 128 of up to 1024
int f32_grid() { return sm_count(); }

cudaError_t launch_f32(Params p, int grid, cudaStream_t s) {
    p.tile_log2 = kTileLog2;
    p.unit_cost = 2;
    const size_t smem = smem_bytes(p.a.D);
    auto kern = p.a.D > 64 ? tree_attention_f32<true> : tree_attention_f32<false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, kThreads, smem, s, p);
}

}  // namespace attn
}  // namespace dspark
