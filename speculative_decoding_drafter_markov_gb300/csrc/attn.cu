// attn.cu -- attention of drafted rows over a paged cache: the general CUDA-core
// kernel (the shapes that neither the tensor-core kernel nor the fp32 one takes),
// the choice among the three and the join of the pieces of a unit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn_common.cuh"

namespace dspark {
namespace attn {

namespace {

// ---------------------------------------------------------------- CUDA cores
// A unit of 16 lines (4 per warp) over tiles of 32 tokens; keys and values of a
// tile are staged in shared memory as fp32 and shared by the lines.  A thread
// scores one line against four tokens, then each warp adds its four lines'
// weighted values, the lanes side by side over D.  Bound by its instructions: 64 caches
// of up to 8192 tokens, 36 lines on each of 8 heads of 128, bf16: 1351 us, against 127 us
// on the tensor cores; one row over 2047 tokens 28 against 12.5.
constexpr int kLines = kSimtLines, kTileLog2 = 5, kTile = 1 << kTileLog2, kThreads = 128;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}

__host__ __device__ inline int padded(int D) { return (D + 3) / 4 * 4; }
inline size_t smem_bytes(int D) {
    const int d = padded(D);
    return sizeof(float) * ((size_t)kLines * d + (size_t)kTile * (d + 4) + (size_t)kTile * d + kLines * kTile);
}

template <typename T, int kDV>  // kDV: float4 columns per lane, ceil(D / 128)
__global__ void __launch_bounds__(kThreads) tree_attention_simt(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) float sh[];
    __shared__ Share shared_share;
    const dspark_tree_attention_args &a = p.a;
    const int D = a.D, DP = padded(D), KS = DP + 4;
    float *sq = sh, *sk = sq + kLines * DP, *sv = sk + kTile * KS, *sp = sv + kTile * DP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int line = tid >> 3, tx = tid & 7;  // scores: this thread's line and its tokens tx + 8 i
    after_predecessor();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        const Share s = share_of(p);
        if (lane == 0) shared_share = s;
    }
    __syncthreads();
    Walk walk(p, shared_share);
    if (tid == 0) p.join[blockIdx.x].pieces = 0;
    Piece x;
    while (walk.next(x)) {
        __syncthreads();
        // the lines' queries, zero beyond them
        const int h = x.head / p.subs, head0 = h * p.G + x.head % p.subs * p.heads, heads = min(p.heads, (h + 1) * p.G - head0);
        for (int i = tid; i < kLines * DP; i += kThreads) {
            const int l = i / DP, d = i % DP, jj = l / p.heads, g = l % p.heads;
            float v = 0.f;
            if (jj < x.n && g < heads && d < D)
                v = to_f32(static_cast<const T *>(a.q)[(x.row0 + x.first + jj) * a.q_row + (head0 + g) * a.q_head + d]);
            sq[l * DP + d] = v;
        }
        const int j = x.first + line / p.heads;  // the scored line's row in its request
        const bool live = line / p.heads < x.n;
        const uint64_t *words = a.mask && live ? a.mask + (size_t)(x.row0 + j) * a.W : nullptr;
        float m = -INFINITY, l = 0.f;
        float4 acc[4][kDV];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < kDV; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);

        for (int t = x.t0; t < x.t1; ++t) {
            const int tok0 = t * kTile;
            __syncthreads();
            // keys and values of the tile, zero beyond the unit's tokens
            const T *kc = static_cast<const T *>(a.k_cache), *vc = static_cast<const T *>(a.v_cache);
            const int per = DP / 4;
            for (int i = tid; i < kTile * per; i += kThreads) {
                const int tk = i / per, d = i % per * 4, tok = tok0 + tk;
                float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
                if (tok < x.tokens) {
                    const int in_table = p.page.of(tok);
                    int pg = a.table[(size_t)x.r * a.max_pages + in_table];
                    if (pg < 0 || pg >= a.n_pages) {
                        set_err(a.err, DSPARK_ERR_RANGE);
                        pg = 0;
                    }
                    const size_t at = (((size_t)pg * a.H + h) * a.page + (tok - in_table * a.page)) * D + d;
                    if (p.vec) {
                        kv = load4(kc + at);
                        vv = load4(vc + at);
                    } else {
                        kv.x = to_f32(kc[at]);
                        vv.x = to_f32(vc[at]);
                        if (d + 1 < D) kv.y = to_f32(kc[at + 1]), vv.y = to_f32(vc[at + 1]);
                        if (d + 2 < D) kv.z = to_f32(kc[at + 2]), vv.z = to_f32(vc[at + 2]);
                        if (d + 3 < D) kv.w = to_f32(kc[at + 3]), vv.w = to_f32(vc[at + 3]);
                    }
                }
                *reinterpret_cast<float4 *>(sk + tk * KS + d) = kv;
                *reinterpret_cast<float4 *>(sv + tk * DP + d) = vv;
            }
            __syncthreads();
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int d = 0; d < DP; d += 4) {
                const float4 q4 = *reinterpret_cast<const float4 *>(sq + line * DP + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(sk + (tx + 8 * i) * KS + d);
                    s[i] = fmaf(q4.x, k4.x, fmaf(q4.y, k4.y, fmaf(q4.z, k4.z, fmaf(q4.w, k4.w, s[i]))));
                }
            }
            const bool tail = tok0 + kTile > x.len;  // rows of this cycle, or tokens beyond the unit's
            bool see[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rel = tok0 + tx + 8 * i - x.len;
                see[i] = rel < 0 || (rel < x.rows && (words ? ((words[rel >> 6] >> (rel & 63)) & 1) : !a.mask && rel <= j));
                s[i] = see[i] ? s[i] * p.scale_log2 : -INFINITY;
            }
            // a NaN score stays one: the maximum skips it, its weight is NaN
            float mt = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
            const float mn = fmaxf(m, mt), ref = mn == -INFINITY ? 0.f : mn;
            const float keep = ex2(m - ref);  // m = -inf: 0
            float w[4], sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = ex2(s[i] - ref);
                sum += w[i];
                // what the line does not see is marked, so that its value is left out below
                sp[line * kTile + tx + 8 * i] = see[i] ? w[i] : -1.f;
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l = fmaf(l, keep, sum);
            m = mn;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = __shfl_sync(0xffffffffu, keep, 8 * i);
#pragma unroll
                for (int c = 0; c < kDV; ++c) {
                    acc[i][c].x *= f;
                    acc[i][c].y *= f;
                    acc[i][c].z *= f;
                    acc[i][c].w *= f;
                }
            }
            const float *wp = sp + 4 * warp * kTile;
            for (int tk = 0; tk < kTile; ++tk) {
                float pw[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) pw[i] = wp[i * kTile + tk];
#pragma unroll
                for (int c = 0; c < kDV; ++c) {
                    const int d = 4 * lane + 128 * c;
                    if (d >= DP) break;
                    const float4 v = *reinterpret_cast<const float4 *>(sv + tk * DP + d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (tail && pw[i] < 0.f) continue;
                        acc[i][c].x = fmaf(pw[i], v.x, acc[i][c].x);
                        acc[i][c].y = fmaf(pw[i], v.y, acc[i][c].y);
                        acc[i][c].z = fmaf(pw[i], v.z, acc[i][c].z);
                        acc[i][c].w = fmaf(pw[i], v.w, acc[i][c].w);
                    }
                }
            }
            __syncwarp();
        }

#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ln = 4 * warp + i, jj = ln / p.heads, g = ln % p.heads;
            const float mm = __shfl_sync(0xffffffffu, m, 8 * i), ll = __shfl_sync(0xffffffffu, l, 8 * i);
            if (jj >= x.n || g >= heads) continue;
            const size_t orow = (size_t)(x.row0 + x.first + jj) * a.Hq + head0 + g;
            const size_t prow = (size_t)(x.slot < 0 ? 0 : x.slot) * p.lines + ln;
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
            for (int c = 0; c < kDV; ++c) {
                const float v[4] = {acc[i][c].x, acc[i][c].y, acc[i][c].z, acc[i][c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int d = 4 * lane + 128 * c + e;
                    if (d >= D) break;
                    if (x.slot < 0) store_out(p, orow * D + d, v[e] * inv);
                    else p.part_o[prow * p.stride + d] = v[e];
                }
            }
            if (lane == 0) {
                if (x.slot >= 0) p.part_ml[prow] = make_float2(mm, ll);
                else if (a.lse) a.lse[orow] = lse_of(mm, ll);
            }
        }
        if (tid == 0 && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
    }
}

// ---------------------------------------------------------------- join
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over a unit's partials.
// At most one unit starts in a CTA and ends in a later one, so CTAs (c, ..) join the
// lines of CTA c's unit: a warp a line, or, where that takes fewer rounds (many pieces
// and few lines, as of one long cache over the whole GPU), the four warps of a CTA share
// a line's pieces.  (Always sharing above eight pieces: 434 lines on 4 heads, 5 caches of
// up to 1312 tokens took 41 us, by rounds 24.)  Bound by latency: partials that are still
// in L2, four under way before the weights are known (eight take the registers of half of
// the CTAs: 2 us more for 256 lines).  About 3 us for a few lines, 9 us for 256 lines in
// each of 16 requests.
constexpr int kJoinWarps = 4, kAhead = 4;

// four (or, E = 1, one) adjacent floats per lane
template <int E>
struct Cells {
    float v[E];
    __device__ __forceinline__ void load(const float *p) {
        if (E == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            v[0] = q.x, v[E > 1 ? 1 : 0] = q.y, v[E > 2 ? 2 : 0] = q.z, v[E > 3 ? 3 : 0] = q.w;
        } else {
            v[0] = *p;
        }
    }
};

// kCols: groups of 32 E columns that a line has
template <int E, int kCols>
__global__ void __launch_bounds__(32 * kJoinWarps, 8) tree_attention_join(const __grid_constant__ Params p) {
    __shared__ float sum_o[kJoinWarps - 1][32 * E * kCols];
    after_predecessor();  // the partials are written
    const Join n = p.join[blockIdx.x];
    if (n.pieces == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.stride;
    // rounds of kAhead partials, and one for the weights, either way
    const int y = gridDim.y, turns = (n.lines + y - 1) / y, turns_warp = (n.lines + y * kJoinWarps - 1) / (y * kJoinWarps);
    const bool many = turns * ((n.pieces + kAhead * kJoinWarps - 1) / (kAhead * kJoinWarps) + 1) <
                      turns_warp * ((n.pieces + kAhead - 1) / kAhead + 1);
    // partial i: the first one, then the first partials of the CTAs after it
    auto slot = [&](int i, int ln) { return (size_t)(i == 0 ? n.first : 2 * ((int)blockIdx.x + i)) * p.lines + ln; };
    const int step = many ? kJoinWarps : 1;  // pieces of this warp: own, own + step, ..
    const int own = many ? warp : 0;
    for (int ln = many ? blockIdx.y : blockIdx.y * kJoinWarps + warp; ln < n.lines; ln += many ? gridDim.y : gridDim.y * kJoinWarps) {
        const int jj = ln / p.heads, g = ln - jj * p.heads;
        if (g >= n.heads) continue;
        float2 ml = lane < n.pieces ? p.part_ml[slot(lane, ln)] : make_float2(-INFINITY, 0.f);
        Cells<E> next[kAhead][kCols];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                const float *from = p.part_o + slot(i, ln) * D;
#pragma unroll
                for (int c = 0; c < kCols; ++c)
                    if (i < n.pieces && E * (lane + 32 * c) < D) next[u][c].load(from + E * (lane + 32 * c));
            }
        };
        fetch(own);
        float M = ml.x;
        for (int i = 32 + lane; i < n.pieces; i += 32) M = fmaxf(M, p.part_ml[slot(i, ln)].x);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        const float ref = M == -INFINITY ? 0.f : M;
        float o[kCols][E], w = ex2(ml.x - ref), L = w * ml.y;
        for (int i = 32 + lane; i < n.pieces; i += 32) {
            const float2 x = p.part_ml[slot(i, ln)];
            L = fmaf(ex2(x.x - ref), x.y, L);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) o[c][e] = 0.f;
        int chunk = 0;  // w is the weight of piece chunk + lane
        for (int i0 = own; i0 < n.pieces; i0 += kAhead * step) {
            if (i0 != own) fetch(i0);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * step;
                if (i >= n.pieces) break;
                if (i >= chunk + 32) {
                    chunk = i & ~31;
                    w = chunk + lane < n.pieces ? ex2(p.part_ml[slot(chunk + lane, ln)].x - ref) : 0.f;
                }
                const float wi = __shfl_sync(0xffffffffu, w, i - chunk);
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (E * (lane + 32 * c) < D) o[c][e] = fmaf(wi, next[u][c].v[e], o[c][e]);
            }
        }
        if (many) {
            __syncthreads();
            if (warp > 0) {
#pragma unroll
                for (int c = 0; c < kCols; ++c)
#pragma unroll
                    for (int e = 0; e < E; ++e) sum_o[warp - 1][E * (lane + 32 * c) + e] = o[c][e];
            }
            __syncthreads();
            if (warp > 0) continue;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int x = 0; x < kJoinWarps - 1; ++x) o[c][e] += sum_o[x][E * (lane + 32 * c) + e];
        }
        const size_t at = (size_t)(n.row + jj) * p.a.Hq + n.head + g;
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int place = E * (lane + 32 * c) + e, d = p.mixed ? plain_column(place) : place;
                if (place < D && d < p.a.D) store_out(p, at * p.a.D + d, o[c][e] * inv);
            }
        if (p.a.lse && lane == 0) p.a.lse[at] = lse_of(M, L);
    }
}

template <typename T, int kDV>
cudaError_t launch_as(const Params &p, int grid, size_t smem, cudaStream_t s) {
    auto kern = tree_attention_simt<T, kDV>;
    if (smem > 32 * 1024) {  // well below the 48 KB, which the kernel's own variables share
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    return launch_close(kern, grid, kThreads, smem, s, p);
}

// CTAs of the CUDA-core kernel that fit an SM's shared memory (capped by its threads)
int simt_grid(int D) {
    const int fit = (int)(220 * 1024 / (smem_bytes(D) + 1024));
    return sm_count() * (fit < 1 ? 1 : fit > 8 ? 8 : fit);
}

}  // namespace

size_t workspace_bytes(int grid, int lines, int stride) {
    return align256(sizeof(Join) * grid) + align256(sizeof(float2) * 2 * (size_t)grid * lines) +
           align256(sizeof(float) * 2 * (size_t)grid * lines * stride);
}

void carve(Params &p, void *ws, int grid) {
    char *c = static_cast<char *>(ws);
    p.join = reinterpret_cast<Join *>(c);
    c += align256(sizeof(Join) * grid);
    p.part_ml = reinterpret_cast<float2 *>(c);
    c += align256(sizeof(float2) * 2 * (size_t)grid * p.lines);
    p.part_o = reinterpret_cast<float *>(c);
}

cudaError_t launch_join(const Params &p, int grid, cudaStream_t s) {
    // a CTA for every line of a unit, as far as the host knows them; the first launch lets
    // them come up while it runs
    const long long lines = (long long)p.a.max_rows * p.heads;
    unsigned y = (unsigned)(lines < 1 ? 1 : lines < p.lines ? lines : p.lines);
    if (y > 32) y = 32;
    auto kern = p.stride % 4 == 0 ? (p.stride <= 128 ? tree_attention_join<4, 1> : tree_attention_join<4, 2>)
                                  : (p.stride <= 64 ? tree_attention_join<1, 2> : tree_attention_join<1, 8>);
    return launch_close(kern, dim3(grid, y), 32 * kJoinWarps, 0, s, p);
}

}  // namespace attn

size_t tree_attention_ws_bytes(const dspark_tree_attention_args &a) {
    // enough for either kernel: which one runs also depends on the pointers
    const size_t simt = attn::workspace_bytes(attn::simt_grid(a.D), attn::kLines, a.D);
    if (a.dtype != DSPARK_BF16 || a.D > 128 || a.Hq / a.H > 128) return simt;
    int block_rows, lines, stride;
    attn::tc_shape(a, &block_rows, &lines, &stride);
    const size_t tc = attn::workspace_bytes(sm_count(), lines, stride);
    return tc > simt ? tc : simt;
}

cudaError_t launch_tree_attention(const dspark_tree_attention_args &a, void *ws, cudaStream_t s) {
    using namespace attn;
    if (sm_count() < 1) return cudaErrorNoDevice;  // the work is cut by the SMs there are
    Params p{};
    p.a = a;
    p.H = a.H;
    p.G = a.Hq / a.H;
    p.masked = a.mask != nullptr;
    p.scale_log2 = a.scale * kLog2e;
    if (tc_supported(a)) {
        p.heads = p.G;
        p.subs = 1;
        tc_shape(a, &p.block_rows, &p.lines, &p.stride);
        p.mixed = 1;
        const int grid = sm_count();
        carve(p, ws, grid);
        cudaError_t e = launch_tc(p, grid, s);
        return e == cudaSuccess ? launch_join(p, grid, s) : e;
    }
    p.heads = p.G < kLines ? p.G : kLines;
    p.subs = (p.G + p.heads - 1) / p.heads;
    p.block_rows = kLines / p.heads;
    p.lines = p.block_rows * p.heads;
    p.stride = a.D;
    p.small_rows = p.block_rows;
    p.small_places = p.large_places = div_by(1);
    p.page = div_by(a.page);
    if (f32_supported(a)) {
        const int grid = f32_grid();
        p.ctas = div_by(grid);
        carve(p, ws, grid);
        cudaError_t e = launch_f32(p, grid, s);
        return e == cudaSuccess ? launch_join(p, grid, s) : e;
    }
    p.tile_log2 = kTileLog2;
    p.unit_cost = 1;
    const int es = a.dtype == DSPARK_BF16 ? 2 : 4;
    p.vec = a.D % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache)) & (4 * es - 1)) == 0;
    const int grid = simt_grid(a.D);
    p.ctas = div_by(grid);
    carve(p, ws, grid);
    const size_t smem = smem_bytes(a.D);
    const bool wide = a.D > 128;
    cudaError_t e;
    if (a.dtype == DSPARK_BF16)
        e = wide ? launch_as<__nv_bfloat16, 2>(p, grid, smem, s) : launch_as<__nv_bfloat16, 1>(p, grid, smem, s);
    else
        e = wide ? launch_as<float, 2>(p, grid, smem, s) : launch_as<float, 1>(p, grid, smem, s);
    if (e != cudaSuccess) return e;
    return launch_join(p, grid, s);
}

}  // namespace dspark
