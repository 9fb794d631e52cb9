// attn_tc.cu -- attention of drafted rows over a paged cache on the 5th-generation
// tensor cores (bf16, D a multiple of 8 up to 128, pages of a multiple of 8 tokens).
//
// A unit's lines (rows x query heads of a group) fill one or two 128-row MMA
// operands.  Per operand and tile of 128 tokens:
//     S = Q K^T   (Q, K in shared memory, S in tensor memory, fp32)
//     P = 2^(S scale log2(e) - m)   rounded to bf16 over S's columns
//     O += P V    (P in tensor memory, V in shared memory as the MN-major operand)
// Two streams, each with its own S and O and four softmax warps, run side by side:
// with two operands a stream per operand, both over every tile; with one, the
// streams take the even and the odd tiles and are added at the end like two
// partials.  The softmax works and hands P over in halves, so that the first half's
// product runs while the second half is formed.  The maximum m is only moved, and O
// rescaled in tensor memory, when a half exceeds it by 2^8 (any reference gives
// the same result; P stays below 2^8 and the fp32 sums far from overflow): the
// running-maximum softmax of Milakov and Gimelshein (arXiv 1805.02867) with a
// reference that may lag behind.
//
// P is rounded to one bf16 term (the MMA wants A in the type of B, the values): against
// 64 bits the outputs are off by 0.0022 to 0.0023 of their size, the rounding of the output
// alone by 0.0017.  A second term, the rest of P in the half of S's columns that the first
// leaves free, brings that to 0.0017, but doubles the second product and a third of
// the softmax, both in the chain that bounds a tile: 64 caches of up to 8192 tokens 146
// instead of 126 us, 16 of up to 16384 with trees of up to 64 rows 126 instead of 98, 8 of
// up to 131072 with up to 256 lines 587 instead of 433, and with 68 lines 433 instead of 420.
//
// Warps 0-7 softmax, 8 and 10 copy keys and values by TMA, a box per page piece,
// through one ring of slots in the order of their use, 9 copies Q and issues the
// MMAs, 11 walks the CTA's share of the work and hands out its pieces.
//
// Bound by HBM while lines are few: a tile of D = 128 is 64 KB, 2,900 clocks of an
// SM's share of the bandwidth, against 1,030 of MMA per operand.  8 heads of 128, bf16:
// 8 caches of up to 131072 tokens with up to 68 lines take 424 us (6.8 TB/s), 64 of up to
// 8192 with up to 36 lines 127 us (5.6 TB/s, the rest starts and ends of pieces), one row
// over 2047 tokens 12.5 us (latency).  With many lines by the chain from S through the
// softmax to P: 8 caches of up to 131072 with up to 256 lines 435 us, 0.88 PFLOP/s.
// S in half tiles of 64 tokens, to give the softmax its first half earlier, took 4 % more
// than whole tiles: an MMA of 64 columns takes 55 clocks, one of 128 takes 64.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <mutex>

#include "attn_common.cuh"
#include "attn_tc.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kThreads = 384, kTileLog2 = 7, kTile = 1 << kTileLog2;
constexpr float kSlack = 8.f;  // log2 by which half a tile may exceed the reference
constexpr int kQueue = 4;      // pieces handed out ahead
// Places in the line of units: of a tile for one operand and for two, tiles' worth of a
// unit's start and end.  With 3 : 5 : 3 the 16 trees of up to 64 rows over up to 16384
// tokens took 100 us, with 1 : 1 : 3 112, with 2 : 4 : 3 106, with 2 : 3 : 3 101.
constexpr int kTilePlaces = 3, kDualPlaces = 5, kUnitCost = 3;

// DP: D padded to the copied width, NQ: operands a unit may have
template <int DP_, int NQ_>
struct Shape {
    static constexpr int DP = DP_, NQ = NQ_;
    static constexpr int kCols = DP / 64;        // a row is copied in blocks of 64 columns
    static constexpr int kBlock = 128 * 128;     // 128 rows of 64 bf16
    static constexpr int kSlot = kCols * kBlock;
    static constexpr int NS = DP == 128 ? 7 - NQ : 12;  // ring slots: what 227 KB hold beside Q
    static constexpr int kOffRing = NQ * kSlot;
    static constexpr int kOffMl = kOffRing + NS * kSlot;    // float2 [2][128]
    static constexpr int kOffPiece = kOffMl + 2 * 128 * 8;  // Piece [kQueue], 64 bytes each
    static constexpr int kOffBar = kOffPiece + 64 * kQueue;
    static constexpr int kBars = 2 * NS + 13 + 2 * kQueue;
    static constexpr int kOffBad = kOffBar + 8 * kBars;     // uint32 [3][8]
    static constexpr int kOffMisc = kOffBad + 96;           // tmem slot, abort flag
    static constexpr int kSmem = kOffMisc + 8;
};
static_assert(sizeof(Piece) <= 64, "a piece's place in the queue");

struct TcParams {
    Params p;
    int op_rows;  // rows of one operand
    int inv_group;  // ceil(2^16 / G): line * inv_group >> 16 = line / G below 256
    int box;      // tokens of a TMA box: a power of two that divides a page
};

// A role's bounded waits.  The first that runs out ends the role (every role
// comes to the CTA's last barrier; the error word tells).  Hundreds of short
// waits make up a piece, so the limit is counted in SM clocks, which cost less to
// read than the wall clock, and only after a run of tries.
constexpr long long kWaitClocks = 4000000000ll;  // about 2 s
struct Waiter {
    volatile int *abort_flag;
    int32_t *err;
    __device__ __forceinline__ bool one(uint64_t *bar, uint32_t parity) const {
        if (tc::mbar_try_wait(bar, parity)) return true;
        return slow(bar, parity);
    }
    __device__ __noinline__ bool slow(uint64_t *bar, uint32_t parity) const {
        const long long t0 = clock64();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (tc::mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (clock64() - t0 > kWaitClocks) break;
        }
        *abort_flag = 1;
        set_err(err, DSPARK_ERR_TIMEOUT);
        return false;
    }
    // by a whole warp, its first lane looking
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
        int ok = 1;
        if ((threadIdx.x & 31) == 0) ok = one(bar, parity) ? 1 : 0;
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    }
};

// The queue of pieces: each reader takes a copy and gives the place back.
struct Queue {
    const Piece *items;
    uint64_t *full, *empty;
    uint32_t n;
    __device__ __forceinline__ bool read_one(const Waiter &w, Piece &x) {
        const int i = n % kQueue;
        if (n > 0 && !w.one(&full[i], (n / kQueue) & 1u)) return false;  // the first is there
        x = *reinterpret_cast<const Piece *>(reinterpret_cast<const char *>(items) + 64 * i);
        tc::mbar_arrive(&empty[i]);
        ++n;
        return x.r >= 0;
    }
    __device__ __forceinline__ bool read_warp(const Waiter &w, Piece &x) {
        const int i = n % kQueue;
        if (n > 0 && !w.warp(&full[i], (n / kQueue) & 1u)) return false;
        x = *reinterpret_cast<const Piece *>(reinterpret_cast<const char *>(items) + 64 * i);
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&empty[i]);
        ++n;
        return x.r >= 0;
    }
};
constexpr int kReaders = 11;  // two copy warps, the MMA warp, eight softmax warps

// where a piece's tiles stand in the ring, counted from the piece's first slot:
// K0 K1 V0 K2 V1 K3 .., or with two operands K0 V0 K1 V1 ..
__device__ __forceinline__ uint32_t key_place(int t, bool dual) { return dual ? 2 * t : t < 2 ? t : 2 * t - 1; }
__device__ __forceinline__ uint32_t value_place(int t, int n, bool dual) { return dual ? 2 * t + 1 : t + min(t + 2, n); }

// 32 mask bits of a row from bit position pos on (its words; beyond `rows` clear)
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
// cycle; negative: the cache) row j sees
__device__ __forceinline__ uint32_t seen_bits(const uint32_t *words, int n_words, int rel0, int rows, int j) {
    if (rel0 + 31 < 0) return 0xffffffffu;
    if (!words) {
        const int n = j - rel0 + 1;  // a chain
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
    }
    if (rel0 >= 0) return mask_bits(words, n_words, rel0, rows);
    return (mask_bits(words, n_words, 0, rows) << -rel0) | ((1u << -rel0) - 1);
}

// 4 x 4 transposition among the four lanes of a quad: a[i] of lane j <-> a[j] of lane i
__device__ __forceinline__ void transpose_quad(uint32_t (&a)[4], int j) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, j & 1 ? a[i] : a[i + 1], 1);
        if (j & 1) a[i] = r;
        else a[i + 1] = r;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, j & 2 ? a[i] : a[i + 2], 2);
        if (j & 2) a[i] = r;
        else a[i + 2] = r;
    }
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&two);
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams tp) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const Params &p = tp.p;
    const dspark_tree_attention_args &a = p.a;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *empty = full + C::NS;
    uint64_t *s_full = empty + C::NS, *p_ready = s_full + 2;  // [stream]; [stream][half]
    uint64_t *half_done = p_ready + 4, *q_full = half_done + 2, *o_free = q_full + 1, *both = o_free + 1,
             *drain = both + 1, *o_last = drain + 1;
    uint64_t *queue_full = o_last + 1, *queue_empty = queue_full + kQueue;
    Piece *pieces = reinterpret_cast<Piece *>(smem + C::kOffPiece);
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    Piece x;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tc::smem_u32(smem) & 1023u) {  // the swizzled tiles need it; the launch gives it
        after_predecessor();
        if (tid == 0) set_err(a.err, DSPARK_ERR_UNSUPPORTED);
        return;
    }
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    } else if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(&s_full[0], 1);
        tc::mbar_init(&s_full[1], 1);
        tc::mbar_init(&half_done[0], 1);
        tc::mbar_init(&half_done[1], 1);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&p_ready[i], 4);
        tc::mbar_init(q_full, 1);
        tc::mbar_init(o_free, 8);
        tc::mbar_init(both, 8);
        tc::mbar_init(drain, 1);
        tc::mbar_init(o_last, 1);
        for (int i = 0; i < kQueue; ++i) {
            tc::mbar_init(&queue_full[i], 1);
            tc::mbar_init(&queue_empty[i], kReaders);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    } else if (warp == 1) {
        if (lane < 24) bad[lane] = 0;
    } else if (warp == 8 && lane == 0) {
        tc::prefetch_tmap(&tmQ);
        tc::prefetch_tmap(&tmK);
        tc::prefetch_tmap(&tmV);
    }
    after_predecessor();  // nothing of the inputs or the workspace was touched so far
    // the table on its way to L2, where it is small, while the CTAs find their shares
    if (warp == 10 && a.R * (long long)a.max_pages <= 32ll * 32 * gridDim.x) {
        const int line = 32 * (blockIdx.x * 32 + lane);
        if (line < a.R * a.max_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + line));
    }
    const Waiter wait{abort_flag, a.err};
    if (warp == 11) {
        // ------------------------------------------------------------ the walk
        // The first piece is handed out by the CTA's barrier, the others by the queue.
        const Share share = share_of(p);
        Walk walk(p, share);
        if (lane == 0) p.join[blockIdx.x].pieces = 0;
        bool more = true;
        for (uint32_t n = 0; more; ++n) {
            more = walk.next(x);
            if (!more) x.r = -1;
            const int i = n % kQueue;
            if (n > 0 && !wait.warp(&queue_empty[i], ((n / kQueue) & 1u) ^ 1u)) break;
            if (lane == 0) *reinterpret_cast<Piece *>(reinterpret_cast<char *>(pieces) + 64 * i) = x;
            if (n == 0) __syncthreads();
            if (lane == 0) {
                tc::mbar_arrive(&queue_full[i]);
                if (more && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
            }
        }
    } else {
        __syncthreads();
    }
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Queue queue{pieces, queue_full, queue_empty, 0};
    uint32_t next = 0, mine = 0;  // copy warps: the slot after the last copy; bit k: slot next - 1 - k was this warp's

    if (warp == 11) {
        // the walk is done
    } else if (warp == 8 || warp == 10) {
        // ------------------------------------------------------------ keys; values
        const bool values = warp == 10;
        const CUtensorMap *map = values ? &tmV : &tmK;
        uint32_t base = 0;  // slots before the piece
        // a lane copies one block of columns of one box
        const int bx = lane / C::kCols, col = lane % C::kCols;
        while (queue.read_warp(wait, x)) {
            const bool dual = C::NQ == 2 && x.n > tp.op_rows;
            const int n = x.t1 - x.t0;
            const int32_t *table = a.table + (size_t)x.r * a.max_pages;
            const int last_tok = x.tokens - 1;
            int in_table = 0;  // of the lane's box
            auto page_at = [&](int t) { return table[in_table = p.page.of(lookup_token(t, kTileLog2, bx, tp.box, last_tok))]; };
            int pg = page_at(x.t0);
            bool ok = true;
            for (int t = 0; t < n; ++t) {
                const int tok0 = (x.t0 + t) * kTile, tok = tok0 + bx * tp.box;
                const int boxes = (min(kTile, x.tokens - tok0) + tp.box - 1) / tp.box;
                const uint32_t pos = base + (values ? value_place(t, n, dual) : key_place(t, dual));
                const int slot = pos % C::NS;
                int go = 1;
                if (lane == 0) {
                    go = wait.one(&empty[slot], ((pos / C::NS) & 1u) ^ 1u) ? 1 : 0;
                    if (go) tc::mbar_expect_tx(&full[slot], (uint32_t)(boxes * tp.box * 128 * C::kCols));
                }
                ok = __shfl_sync(0xffffffffu, go, 0) != 0;
                if (!ok) break;
                mine = (pos + 1 - next < 32 ? mine << (pos + 1 - next) : 0u) | 1u;
                next = pos + 1;
                if (bx < boxes) {
                    if (pg < 0 || pg >= a.n_pages) {
                        set_err(a.err, DSPARK_ERR_RANGE);
                        pg = 0;
                    }
                    tc::tma_load_3d(smem + C::kOffRing + slot * C::kSlot + col * C::kBlock + bx * tp.box * 128, map,
                                    &full[slot], 64 * col, tok - in_table * a.page, pg * a.H + x.head);
                }
                __syncwarp();
                if (t + 1 < n) pg = page_at(x.t0 + t + 1);
            }
            if (!ok) break;
            base += 2 * n;
        }
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------------ Q and the MMAs
        if (lane == 0) {
            constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, kTile);
            constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, C::DP) | tc::kIdescBMnMajor;
            const uint32_t sbase = tc::smem_u32(smem);
            const uint32_t q_lo = tc::desc_lo_k128(sbase), k_lo = tc::desc_lo_k128(sbase + C::kOffRing),
                           v_lo = tc::desc_lo_mn128(sbase + C::kOffRing, C::kBlock);
            uint32_t q_loads = 0, done = 0, p_phase[2] = {0, 0};
            int slot = 0, kslot = 0, vslot = 0;
            uint32_t phase = 0;  // of the next slot
            auto load_q = [&](const Piece &y) {
                const int ops = C::NQ == 2 && y.n > tp.op_rows ? 2 : 1;
                tc::mbar_expect_tx(q_full, (uint32_t)(ops * tp.op_rows * p.G * 128 * C::kCols));
                for (int o = 0; o < ops; ++o)
                    for (int col = 0; col < C::kCols; ++col)
                        tc::tma_load_3d(smem + o * C::kSlot + col * C::kBlock, &tmQ, q_full, 64 * col, y.head * p.G,
                                        y.row0 + y.first + o * tp.op_rows);
                ++q_loads;
            };
            auto next_slot = [&](int &mine) {
                mine = slot;
                const bool got = wait.one(&full[slot], phase);
                if (++slot == C::NS) slot = 0, phase ^= 1u;
                return got;
            };
            bool more = queue.read_one(wait, x), ok = true;
            if (more) load_q(x);
            while (ok && more) {
                const bool dual = C::NQ == 2 && x.n > tp.op_rows;
                const int steps = (x.t1 - x.t0) << (dual ? 1 : 0);
                // a tile's keys and values serve one step, or with two operands the
                // steps of both streams
                auto scores = [&](int w) {
                    if ((!dual || w == 0) && !next_slot(kslot)) return false;
                    tc::tc_fence_after();
                    const uint32_t al = q_lo + (dual && w ? C::kSlot >> 4 : 0), bl = k_lo + kslot * (C::kSlot >> 4);
#pragma unroll
                    for (int kk = 0; kk < C::DP / 16; ++kk) {
                        const uint32_t step = ((kk >> 2) * C::kBlock + (kk & 3) * 32) >> 4;
                        tc::umma_bf16_lo(tmem + 128 * w, al + step, bl + step, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    tc::umma_commit(&s_full[w]);
                    if (!dual || w == 1) tc::umma_commit(&empty[kslot]);
                    return true;
                };
                auto values = [&](int i, int w) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!wait.one(&p_ready[2 * w + half], p_phase[w])) return false;
                        if (half == 0) {
                            if (i == 0 && done > 0 && !wait.one(o_free, (done - 1) & 1u)) return false;
                            if ((!dual || w == 0) && !next_slot(vslot)) return false;
                        }
                        tc::tc_fence_after();
                        const uint32_t bl = v_lo + vslot * (C::kSlot >> 4);
#pragma unroll
                        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                            tc::umma_bf16_ta_lo(tmem + 256 + 128 * w, tmem + 128 * w + 64 * half + 8 * (kk & 3), bl + ((kk * 2048) >> 4), idesc_o,
                                                i >= 2 || kk > 0 ? 1u : 0u);
                        if (half == 0) tc::umma_commit(&half_done[w]);
                    }
                    p_phase[w] ^= 1u;
                    if (!dual || w == 1) tc::umma_commit(&empty[vslot]);
                    if (i + 1 == steps) tc::umma_commit(o_last);
                    return true;
                };
                ok = wait.one(q_full, (q_loads - 1) & 1u) && scores(0) && (steps == 1 || scores(1));
                for (int i = 0; ok && i < steps; i += 2) {
                    ok = values(i, 0) && (i + 2 >= steps || scores(0));
                    if (ok && i + 1 < steps) ok = values(i + 1, 1) && (i + 3 >= steps || scores(1));
                }
                ++done;
                // every S of the piece is done (its P was waited for): Q may go
                if (ok) {
                    more = queue.read_one(wait, x);
                    if (more) load_q(x);
                }
            }
            if (!ok || *abort_flag) {
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
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
        uint32_t count = 0;  // tiles of this stream so far
        uint32_t base = 0, done = 0;
        const uint32_t s_tmem = tmem + quad + 128 * w, o_tmem = tmem + quad + 256 + 128 * w;
        const float scale = fmaxf(p.scale_log2, 1e-37f);  // 0 would make -inf x 0 of what is not seen
        while (queue.read_warp(wait, x)) {
            const bool dual = C::NQ == 2 && x.n > tp.op_rows;
            const int n = x.t1 - x.t0;
            const int row_first = x.first + (dual && w ? tp.op_rows : 0);
            const int lines = (dual ? (w ? x.n - tp.op_rows : tp.op_rows) : x.n) * p.G;
            const int steps = dual ? n : (n + 1 - w) >> 1;
            const bool active = 32 * q < lines, live = row < lines;
            const int jj = (row * tp.inv_group) >> 16, j = row_first + jj;  // row / G
            // rows of the cycle before `base_rel` are seen by every line of the unit
            const int base_rel = a.mask ? 0 : x.first + 1;
            const uint32_t *words = a.mask && live ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + j) * a.W) : nullptr;
            uint32_t *flags = bad + 8 * (done % 3u);
            float m = -INFINITY, l = 0.f;
            bool ok = true;
            for (int u = 0; u < steps; ++u, ++count) {
                const int tl = dual ? u : 2 * u + w;
                const int tok0 = (x.t0 + tl) * kTile;
                const bool tail = tok0 + kTile > x.len + base_rel;
                ok = wait.warp(&s_full[w], count & 1u);
                if (!ok) break;
                tc::tc_fence_after();
                if (tail && (!dual || w == 0)) {
                    // (S of the tile is there, so the copies into this slot before its values
                    // are too.)  Values that some lines do not see must not reach them as 0 x inf:
                    // slots beyond the tokens are zeroed, infinities and NaN of the
                    // cycle's rows too, and those added back below where they are seen.
                    const uint32_t pos = base + value_place(tl, n, dual);
                    const int slot = pos % C::NS;
                    ok = wait.warp(&full[slot], (pos / C::NS) & 1u);
                    if (!ok) break;
                    const int tok = tok0 + row, rel = tok - x.len - base_rel;  // a thread a token
                    if (tok >= x.tokens || rel >= 0) {
                        bool found = false;
                        unsigned char *from = smem + C::kOffRing + slot * C::kSlot + row * 128;
#pragma unroll 1
                        for (int b = 0; b < C::kCols; ++b, from += C::kBlock) {
                            // eight 16-byte pieces, each lane from another one on (the banks)
                            if (tok >= x.tokens) {
#pragma unroll
                                for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4 *>(from + ((c ^ lane) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                                continue;
                            }
                            uint4 v[8];
                            uint32_t hits = 0;
#pragma unroll
                            for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4 *>(from + ((c ^ lane) & 7) * 16);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const uint32_t e[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                                for (int i = 0; i < 4; ++i)  // an exponent of ones carries into the sign's place
                                    hits |= ((e[i] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u;
                            }
                            if (hits == 0) continue;
                            found = true;
#pragma unroll 1
                            for (int i = 0; i < 64; ++i) {
                                unsigned short *at = reinterpret_cast<unsigned short *>(from) + i;
                                if ((*at & 0x7f80u) == 0x7f80u) *at = 0;
                            }
                        }
                        if (found && rel < 256) atomicOr(&flags[rel >> 5], 1u << (rel & 31));
                        tc::fence_proxy_async_smem();
                    }
                }
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t s_half = s_tmem + 64 * half;
                    if (active) {
                        float s[64];
                        tc::tmem_ld32(s_half, s);
                        tc::tmem_ld32(s_half + 32, s + 32);
                        tc::tmem_wait_ld();
                        if (tail) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                // lines beyond the unit's see nothing; what they hold is not read
                                const uint32_t see = live ? seen_bits(words, 2 * a.W, tok0 + 64 * half + 32 * c - x.len, x.rows, j) : 0u;
#pragma unroll
                                for (int i = 0; i < 32; ++i) s[32 * c + i] = see & (1u << i) ? s[32 * c + i] : -INFINITY;
                            }
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 64; i += 4)
#pragma unroll
                            for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], s[i + c]);
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                        if (u == 0 && half == 0) {
                            m = top;
                        } else if (__any_sync(0xffffffffu, top > m + kSlack)) {
                            const float to = top > m + kSlack ? top : m;
                            const float f = to == -INFINITY ? 1.f : ex2(m - to);
                            m = to;
                            l *= f;
                            // the products so far are in O: those of the tile before were
                            // issued before this tile's S, that of the first half says so
                            if (half == 1) ok = wait.warp(&half_done[w], count & 1u);
                            tc::tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < C::DP; c += 16) {
                                uint32_t o[16];
                                tc::tmem_ld16(o_tmem + c, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                tc::tmem_st16(o_tmem + c, o);
                            }
                        }
                        const float ref = m == -INFINITY ? 0.f : m;
                        // two weights at a time: arguments and sums in pairs
                        float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
                        const float2 by = {scale, scale}, off = {-ref, -ref};
                        uint32_t r[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 arg = fma2({s[2 * i], s[2 * i + 1]}, by, off);
                            const float2 e = {ex2(arg.x), ex2(arg.y)};
                            sum[i & 1] = add2(sum[i & 1], e);
                            r[i] = pack(e.x, e.y);
                        }
                        tc::tmem_st32(s_half, r);
                        sum[0] = add2(sum[0], sum[1]);
                        l += sum[0].x + sum[0].y;
                        tc::tmem_wait_st();
                        tc::tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&p_ready[2 * w + half]);
                }
                if (!ok) break;
            }
            if (!ok) break;

            // ---------------------------------------------------------- the piece's end
            // with one operand both streams hold a part of every line
            if (done > 0 && !wait.warp(both, 1u)) break;  // the last piece's ml was read
            ml[128 * w + row] = make_float2(m, l);  // of no tile: -inf, 0
            if (tid < 8) bad[8 * ((done + 1) % 3u) + tid] = 0;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(both);
            if (!wait.warp(both, 0u)) break;
            float f0 = 1.f, f1 = 0.f;
            if (!dual) {
                const float2 s0 = ml[row], s1 = ml[128 + row];
                m = fmaxf(s0.x, s1.x);
                const float ref = m == -INFINITY ? 0.f : m;
                f0 = ex2(s0.x - ref);
                f1 = ex2(s1.x - ref);
                l = fmaf(f0, s0.y, f1 * s1.y);
            }
            uint32_t any_bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) any_bad |= flags[i];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(both);
            if (!wait.warp(o_last, done & 1u)) break;
            tc::tc_fence_after();
            if (active) {
                const bool whole = x.slot < 0;
                const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                f0 *= inv;
                f1 *= inv;
                // with two streams of the same lines each finishes half of the columns
                const int c0 = dual ? 0 : w * (C::DP / 2), c1 = dual ? C::DP : c0 + C::DP / 2;
                const size_t prow0 = (size_t)(whole ? 0 : x.slot) * p.lines + (row_first - x.first) * p.G;
                const bool add = !dual && n > 1;  // one tile: the second stream's O is not this piece's
                const int j4 = lane & 3;
#pragma unroll 1
                for (int rb = 0; rb < 32; rb += 16) {
                    if (32 * q + rb >= lines) break;
                    // the two lines of this lane's elements: factors, place of the output
                    float fa[2], fb[2];
                    bool in[2];
                    int jr[2];
                    __nv_bfloat16 *out[2];
                    float *part[2];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int at = rb + 8 * hf + (lane >> 2), ln = 32 * q + at;
                        fa[hf] = __shfl_sync(0xffffffffu, f0, at);
                        fb[hf] = __shfl_sync(0xffffffffu, f1, at);
                        in[hf] = ln < lines;
                        const int row_in = (ln * tp.inv_group) >> 16, g = ln - row_in * p.G;  // ln / G
                        jr[hf] = row_first + row_in;
                        out[hf] = static_cast<__nv_bfloat16 *>(a.out) + ((size_t)(x.row0 + jr[hf]) * a.Hq + x.head * p.G + g) * a.D + 8 * j4;
                        part[hf] = p.part_o + (prow0 + ln) * p.stride + 4 * j4;
                    }
#pragma unroll 1
                    for (int c = c0; c < c1; c += 32) {
                        const uint32_t from = tmem + quad + ((uint32_t)rb << 16) + 256 + c;
                        float o[16], o1[16];
                        tc::tmem_ld_frag32(from + (dual ? 128 * w : 0), o);
                        if (add) tc::tmem_ld_frag32(from + 128, o1);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= fa[(i >> 1) & 1];
                        if (add) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = fmaf(fb[(i >> 1) & 1], o1[i], o[i]);
                        }
                        if (any_bad) {
#pragma unroll 1
                            for (int hf = 0; hf < 2; ++hf) {
                                if (!in[hf]) continue;
                                const uint32_t *mine = a.mask ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + jr[hf]) * a.W) : nullptr;
#pragma unroll 1
                                for (int b = 0; b < 256; ++b) {
                                    if (!((flags[b >> 5] >> (b & 31)) & 1u)) continue;
                                    const int rel = b + base_rel, tok = x.len + rel;
                                    if (!(seen_bits(mine, 2 * a.W, rel, x.rows, jr[hf]) & 1u)) continue;
                                    int pg = a.table[(size_t)x.r * a.max_pages + tok / a.page];
                                    if (pg < 0 || pg >= a.n_pages) pg = 0;
                                    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_cache) +
                                                             (((size_t)pg * a.H + x.head) * a.page + tok % a.page) * a.D;
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
#pragma unroll
                                        for (int e = 0; e < 2; ++e) {
                                            const int d = c + 8 * k + 2 * j4 + e;
                                            const float val = d < a.D ? __bfloat162float(v[d]) : 0.f;
                                            if (fabsf(val) < INFINITY) continue;
                                            if (hf == 0) o[4 * k + e] += val;
                                            else o[4 * k + 2 + e] += val;
                                        }
                                }
                            }
                            __syncwarp();
                        }
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            if (whole) {
                                uint32_t r[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) r[k] = pack(o[4 * k + 2 * hf], o[4 * k + 2 * hf + 1]);
                                transpose_quad(r, j4);  // now columns c + 8 j4 .. + 7
                                if (in[hf] && c + 8 * j4 < a.D)
                                    *reinterpret_cast<uint4 *>(out[hf] + c) = make_uint4(r[0], r[1], r[2], r[3]);
                            } else if (in[hf]) {
#pragma unroll
                                for (int k = 0; k < 4; k += 2)
                                    *reinterpret_cast<float4 *>(part[hf] + c + 8 * k) =
                                        make_float4(o[4 * k + 2 * hf], o[4 * k + 2 * hf + 1], o[4 * k + 4 + 2 * hf], o[4 * k + 5 + 2 * hf]);
                            }
                        }
                    }
                }
                if (live && (dual || w == 0)) {
                    if (!whole) p.part_ml[prow0 + row] = make_float2(m, l);
                    else if (a.lse) a.lse[(size_t)(x.row0 + j) * a.Hq + x.head * p.G + row - jj * p.G] = lse_of(m, l);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(o_free);
            base += 2 * (uint32_t)n;
            ++done;
        }
        tc::tc_fence_before();
    }
    __syncthreads();
    if (*abort_flag) {
        // A role gave up (else the MMAs have waited for every copy): let the copies
        // land before the CTA's memory goes.  One whose slot was used again is taken
        // for one in flight, and costs the limit of a wait.
        if (lane == 0)
            for (uint32_t k = 0; k < (uint32_t)C::NS; ++k)
                if ((mine >> k) & 1u) tc::mbar_wait_drain(&full[(next - 1 - k) % C::NS], ((next - 1 - k) / C::NS) & 1u, a.err);
        __syncthreads();
    }
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// A bf16 tensor of three dimensions (elements, the first adjacent; strides of the
// other two in bytes) in boxes of 64 elements of the first, 128-byte swizzle; zeros
// beyond the tensor.
bool encode_bf16_map3(CUtensorMap *m, const void *base, const uint64_t (&dims)[3], const uint64_t (&strides)[2],
                      const uint32_t (&box)[3]) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    if (!encode) return false;
    const cuuint64_t d[3] = {dims[0], dims[1], dims[2]};
    const cuuint64_t st[2] = {strides[0], strides[1]};
    const cuuint32_t b[3] = {box[0], box[1], box[2]};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), d, st, b, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    auto kern = tree_attention_tc<C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, kThreads, C::kSmem, s, q, k, v, tp);
}

}  // namespace

bool tc_supported(const dspark_tree_attention_args &a) {
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return a.dtype == DSPARK_BF16 && a.scale >= 0.f && a.D % 8 == 0 && a.D <= 128 && a.page % 8 == 0 && a.Hq / a.H <= 128 && al16(a.q) &&
           al16(a.k_cache) && al16(a.v_cache) && al16(a.out) && a.q_row % 8 == 0 && a.q_head % 8 == 0 && a.q_row > 0 &&
           a.q_head > 0 && a.q_row < (1ll << 38) && a.q_head < (1ll << 38) && tc_available();
}

// One operand while the host's hint says that a request's lines fit it, else two: a unit
// of two reads its keys once for twice the lines.  (8 caches of up to 131072 tokens, up
// to 256 lines: 435 us with two, 572 with one; 4 prompts of up to 4096 rows: 192 and 229;
// 16 caches of up to 1000 tokens, where there are few pieces to share: 33 and 29.)
void tc_shape(const dspark_tree_attention_args &a, int *block_rows, int *lines, int *stride) {
    const int G = a.Hq / a.H, one = 128 / G;
    *block_rows = a.max_rows > one ? 2 * one : one;
    *lines = *block_rows * G;
    *stride = a.D > 64 ? 128 : 64;
}

cudaError_t launch_tc(Params p, int grid, cudaStream_t s) {
    const dspark_tree_attention_args &a = p.a;
    TcParams tp{};
    tp.op_rows = 128 / p.G;
    tp.inv_group = (65536 + p.G - 1) / p.G;
    p.tile_log2 = kTileLog2;
    p.small_rows = tp.op_rows;
    p.small_places = div_by(kTilePlaces);
    p.large_places = div_by(p.block_rows > tp.op_rows ? kDualPlaces : kTilePlaces);
    p.page = div_by(a.page);
    p.ctas = div_by(grid);
    p.unit_cost = kUnitCost;
    tp.p = p;
    tp.box = a.page & -a.page;
    if (tp.box > kTile) tp.box = kTile;
    CUtensorMap q, k, v;
    const uint64_t dims[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.N};
    const uint64_t strides[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_row * 2};
    const uint32_t bx[3] = {64, (uint32_t)p.G, (uint32_t)tp.op_rows};
    if (!encode_bf16_map3(&q, a.q, dims, strides, bx) || !encode_cache(&k, a.k_cache, a, tp.box) ||
        !encode_cache(&v, a.v_cache, a, tp.box))
        return cudaErrorInvalidValue;
    const bool two = p.block_rows > tp.op_rows;
    if (a.D > 64)
        return two ? launch_as<Shape<128, 2>>(tp, grid, q, k, v, s) : launch_as<Shape<128, 1>>(tp, grid, q, k, v, s);
    return two ? launch_as<Shape<64, 2>>(tp, grid, q, k, v, s) : launch_as<Shape<64, 1>>(tp, grid, q, k, v, s);
}

}  // namespace attn
}  // namespace dspark
