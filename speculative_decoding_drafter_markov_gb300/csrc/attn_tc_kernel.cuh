// attn_tc.cuh's wrappers at work: the tensor-core kernel of the attention, for caches in 16
// bits (attn_tc.cu, which says how it works) and in 4 (attn4_tc.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "attn_common.cuh"
#include "attn_tc.cuh"
#include "cache4.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kTileLog2 = 7, kTile = 1 << kTileLog2;
constexpr float kSlack = 8.f;  // log2 by which half a tile may exceed the reference
constexpr int kQueue = 4;      // pieces handed out ahead
// Places in the line of units: of a tile for one operand and for two, tiles' worth of a
// unit's start and end.  With 3 : 5 : 3 the 16 trees of up to 64 rows over up to 16384
// tokens took 100 us, with 1 : 1 : 3 112, with 2 : 4 : 3 106, with 2 : 3 : 3 101.
constexpr int kTilePlaces = 3, kDualPlaces = 5, kUnitCost = 3;

// DP: D padded to the copied width, NQ: operands a unit may have, FOUR: caches in 4 bits
template <int DP_, int NQ_, bool FOUR_ = false>
struct Shape {
    static constexpr int DP = DP_, NQ = NQ_;
    static constexpr bool FOUR = FOUR_;
    // Warps that unpack keys, and as many values.  Two of each leave the softmax 128 registers a thread, which hold a row's
    // 64 scores at once (kHold), four of each 96, and the scores are read twice from tensor memory, 32 at a time.
    // One operand (8 caches of up to 131072 tokens, up to 128 lines): 461 us with two of each, 485 with four.  Two operands want
    // a tile in half the time per line: 16 trees of up to 64 rows 168 and 152.
    static constexpr int kUnpack = NQ == 1 ? 2 : 4;
    static constexpr bool kHold = !FOUR || NQ == 1;
    static constexpr int kThreads = FOUR ? 384 + 64 * kUnpack : 384;
    static constexpr int kReaders = FOUR ? 11 + 2 * kUnpack : 11;  // of pieces: two copy warps, the MMA warp, eight softmax warps, those that unpack
    static constexpr int kCols = DP / 64;        // a row is copied in blocks of 64 columns
    static constexpr int kBlock = 128 * 128;     // 128 rows of 64 16-bit elements
    static constexpr int kSlot = kCols * kBlock;
    // ring slots: what 227 KB hold beside Q, and the packed tiles' ring
    static constexpr int NS = FOUR ? (DP == 128 ? 5 - NQ : 6) : (DP == 128 ? 7 - NQ : 12);
    // packed tiles: a ring for keys and one for values, each filled by one warp and emptied by one
    // group in its order (in a ring for both, a warp that is a round ahead of the other kind
    // would take the phase before for the one that it waits for)
    static constexpr int NP = FOUR ? (DP == 128 ? 3 : 6) : 0;
    static constexpr int kPacked = 128 * DP / 16 * 9;  // codes, then scales, of 128 tokens
    static constexpr int kOffRing = NQ * kSlot;
    static constexpr int kOffPacked = kOffRing + NS * kSlot;
    static constexpr int kOffMl = kOffPacked + 2 * NP * kPacked;  // float2 [2][128]
    static constexpr int kOffPiece = kOffMl + 2 * 128 * 8;    // Piece [kQueue], 64 bytes each
    static constexpr int kOffBar = kOffPiece + 64 * kQueue;
    static constexpr int kBars = 2 * NS + 4 * NP + 13 + 2 * kQueue;
    // The reference that a weight is relative to stands kLift below the maximum: a weight of fp16 is then
    // off by 2^-11 of it, or by 2^-32 of the largest where it is below 2^-21 of that (and zero below
    // 2^-32), and none passes 2^15.  (bf16 would lose 2^-8; the sum is of the weights before they are rounded.)
    static constexpr float kLift = FOUR ? 7.f : 0.f;
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 two = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&two);
}

// The role of the warps that unpack tiles of a cache in 4 bits into the ring, half of them
// keys (kKeys) as the bf16 numbers that they are, half values as the eighths of them in
// fp16 (the whole range of n s, 2^-16 to 401408, is exact there, and the weights beside them
// may be fp16).  A lane has 16 elements of a row, a scale's, per turn.
template <typename C, bool kKeys>
__device__ __forceinline__ void unpack_tiles(unsigned char *smem, const dspark_tree_attention_args &a, int warp, const Waiter &wait,
                                             Queue &queue, uint64_t *copied, uint64_t *copy_free, uint64_t *full, uint64_t *empty,
                                             int op_rows) {
    constexpr int kLanes = C::DP / 16, kRows = 32 / kLanes, kTurns = 8 / kRows;  // lanes of a row, rows of a turn, turns of eight rows
    constexpr int kEights = 16 / C::kUnpack;  // eights of rows of a tile and warp
    const int lane = threadIdx.x & 31, g = lane % kLanes, row = lane / kLanes;
    const bool in = 16 * g < a.D;
    // Lanes of the upper columns write their second piece first, so that eight lanes' pieces fall on all banks; the second
    // turn's rows have bit 2 of the swizzle set.
    const bool flip = C::DP == 128 && g >= 4;
    const int first = (g >> 2) * C::kBlock + row * 128;
    const int piece0 = (((2 * g + (flip ? 1 : 0)) & 7) ^ row) << 4, piece1 = piece0 ^ 16;
    const int code_row = a.D / 2, scale_row = a.D / 16, eight0 = kEights * warp;
    // columns beyond D: zeros in every slot, once
    if (!in) {
#pragma unroll 1
        for (int i = 0; i < C::NS * kEights * kTurns; ++i) {
            const int t = i % kTurns, eight = eight0 + (i / kTurns) % kEights;
            unsigned char *at = smem + C::kOffRing + i / (kEights * kTurns) * C::kSlot + first + eight * 1024 + t * kRows * 128;
            *reinterpret_cast<uint4 *>(at + (piece0 ^ (64 * t))) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4 *>(at + (piece1 ^ (64 * t))) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    uint32_t base = 0;
    Piece x;
    while (queue.read_warp(wait, x)) {
        const bool dual = C::NQ == 2 && x.n > op_rows;
        const int n = x.t1 - x.t0;
        for (int i = 0; i < n; ++i) {
            const uint32_t pos = base + (kKeys ? key_place(i, dual) : value_place(i, n, dual)), item = base / 2 + i;
            const int from = item % C::NP, slot = pos % C::NS;
            if (!wait.warp(&copied[from], (item / C::NP) & 1u)) return;
            const unsigned char *packed = smem + C::kOffPacked + ((kKeys ? 0 : C::NP) + from) * C::kPacked;
            const unsigned char *code = packed + (8 * eight0 + row) * code_row + 8 * g, *scale = packed + kTile * code_row + (8 * eight0 + row) * scale_row + g;
            // (Slots are given back in the ring's order, and items of one kind are three places apart at most, no
            // more than there are slots: the phase before the one waited for has passed.)
            if (!wait.warp(&empty[slot], ((pos / C::NS) & 1u) ^ 1u)) return;
            unsigned char *to = smem + C::kOffRing + slot * C::kSlot + first + eight0 * 1024;
            // Eight rows at a time and no more: the code of all roles has to stay in the SM's first instruction caches (with all 32
            // rows of a warp unrolled four of ten stalls were for instructions, and a tile took twice the time).
#pragma unroll 1
            for (int e8 = 0; e8 < kEights; ++e8) {
                uint2 w[kTurns];
                uint32_t b[kTurns];
#pragma unroll
                for (int t = 0; t < kTurns; ++t) {
                    w[t] = make_uint2(0u, 0u);
                    b[t] = 0;
                    if (in) {
                        w[t] = *reinterpret_cast<const uint2 *>(code + t * kRows * code_row);
                        b[t] = scale[t * kRows * scale_row];
                    }
                }
#pragma unroll
                for (int t = 0; t < kTurns; ++t) {
                    uint32_t r[2][4];
                    const uint32_t word[2] = {flip ? w[t].y : w[t].x, flip ? w[t].x : w[t].y};
                    if (kKeys) {
                        const uint32_t s = b[t] == cache4::kNoNumbers ? 0x7fc07fc0u : cache4::bf16_scales(b[t]);
                        const uint32_t off = cache4::bf16_offset(s);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[h][e] = cache4::bf16_of(word[h], e, s, off);
                    } else {
                        const float s1 = b[t] == cache4::kNoNumbers ? NAN : cache4::eighth_of(b[t]);
                        const uint32_t s = pack_half(s1, s1);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[h][e] = cache4::half_of(word[h] >> (8 * (e >> 1)), e & 1, s);
                    }
                    if (in) {
                        *reinterpret_cast<uint4 *>(to + t * kRows * 128 + (piece0 ^ (64 * t))) = make_uint4(r[0][0], r[0][1], r[0][2], r[0][3]);
                        *reinterpret_cast<uint4 *>(to + t * kRows * 128 + (piece1 ^ (64 * t))) = make_uint4(r[1][0], r[1][1], r[1][2], r[1][3]);
                    }
                }
                code += 8 * code_row;
                scale += 8 * scale_row;
                to += 1024;
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&full[slot]);
                tc::mbar_arrive(&copy_free[from]);
            }
        }
        base += 2 * (uint32_t)n;
    }
}

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1)
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
    // what the copies fill: the packed tiles' rings (keys, values), or the ring itself
    uint64_t *copied = C::FOUR ? queue_empty + kQueue : full, *copy_free = C::FOUR ? copied + 2 * C::NP : empty;
    constexpr int kCopies = C::FOUR ? C::NP : C::NS;
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
            tc::mbar_init(&full[i], C::FOUR ? C::kUnpack : 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2 * C::NP; ++i) {
            tc::mbar_init(&copied[i], 1);
            tc::mbar_init(&copy_free[i], C::kUnpack);
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
            tc::mbar_init(&queue_empty[i], C::kReaders);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    } else if (warp == 1) {
        if (lane < 24) bad[lane] = 0;
    } else if (warp == 8 && lane == 0) {
        tc::prefetch_tmap(&tmQ);
        if (!C::FOUR) {
            tc::prefetch_tmap(&tmK);
            tc::prefetch_tmap(&tmV);
        }
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
        if (C::FOUR && values) copied += C::NP, copy_free += C::NP;
        unsigned char *ring = smem + (C::FOUR ? C::kOffPacked + (values ? C::NP * C::kPacked : 0) : C::kOffRing);
        // a lane copies one block of columns of one box, or its codes or its scales
        constexpr int kParts = C::FOUR ? 2 : C::kCols;
        const int bx = lane / kParts, col = lane % kParts;
        const int row_bytes = C::FOUR ? a.D / 16 * 9 : 128 * C::kCols;
        const unsigned char *cache = static_cast<const unsigned char *>(values ? a.v_cache : a.k_cache);
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
                const uint32_t pos = C::FOUR ? base / 2 + t : base + (values ? value_place(t, n, dual) : key_place(t, dual));
                const int slot = pos % kCopies;
                int go = 1;
                if (lane == 0) {
                    go = wait.one(&copy_free[slot], ((pos / kCopies) & 1u) ^ 1u) ? 1 : 0;
                    if (go) tc::mbar_expect_tx(&copied[slot], (uint32_t)(boxes * tp.box * row_bytes));
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
                    if constexpr (C::FOUR) {
                        // tokens tok .. tok + box - 1: codes or scales of the page's run of bytes
                        const int bytes = col ? a.D / 16 : a.D / 2;
                        const unsigned char *from = cache + ((long long)pg * a.H + x.head) * cache4::page_bytes(a.page, a.D) +
                                                    (col ? cache4::code_bytes(a.page, a.D) : 0) + (long long)(tok - in_table * a.page) * bytes;
                        tc::bulk_load(ring + slot * C::kPacked + (col ? kTile * (a.D / 2) : 0) + bx * tp.box * bytes, from,
                                      (uint32_t)(tp.box * bytes), &copied[slot]);
                    } else {
                        tc::tma_load_3d(ring + slot * C::kSlot + col * C::kBlock + bx * tp.box * 128, map,
                                        &full[slot], 64 * col, tok - in_table * a.page, pg * a.H + x.head);
                    }
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
            constexpr uint32_t idesc_o = (C::FOUR ? tc::idesc_f16_f32(128, C::DP) : tc::idesc_bf16_f32(128, C::DP)) | tc::kIdescBMnMajor;
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
    } else if (C::FOUR && warp >= 12) {
        // ------------------------------------------------------------ 4 bits to 16
        if constexpr (C::FOUR) {
            if (warp < 12 + C::kUnpack) unpack_tiles<C, true>(smem, a, warp - 12, wait, queue, copied, copy_free, full, empty, tp.op_rows);
            else unpack_tiles<C, false>(smem, a, warp - 12 - C::kUnpack, wait, queue, copied + C::NP, copy_free + C::NP, full, empty, tp.op_rows);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, q = warp & 3, row = 32 * q + lane;
        const uint32_t quad = (uint32_t)(32 * q) << 16;
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
        uint32_t count = 0;  // tiles of this stream so far
        uint32_t base = 0, done = 0;
        const uint32_t s_tmem = tmem + quad + 128 * w, o_tmem = tmem + quad + 256 + 128 * w;
        const float scale = fmaxf(p.scale_log2, 1e-37f);  // 0 would make -inf x 0 of what is not seen
        // an exponent of ones, and one in its lowest place, in both halves of a word
        constexpr uint32_t kExponent = C::FOUR ? 0x7c00u : 0x7f80u, kLowest = C::FOUR ? 0x04000400u : 0x00800080u;
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
                                    hits |= ((e[i] & 0x7fff7fffu) + kLowest) & 0x80008000u;
                            }
                            if (hits == 0) continue;
                            found = true;
#pragma unroll 1
                            for (int i = 0; i < 64; ++i) {
                                unsigned short *at = reinterpret_cast<unsigned short *>(from) + i;
                                if ((*at & kExponent) == kExponent) *at = 0;
                            }
                        }
                        if (found && rel < 256) atomicOr(&flags[rel >> 5], 1u << (rel & 31));
                        tc::fence_proxy_async_smem();
                    }
                }
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t s_half = s_tmem + 64 * half;
                    if (C::FOUR && active && tail) {
                        // what a line does not see, and all that lines beyond the unit's hold, becomes -inf before the loop below
#pragma unroll 1
                        for (int c = 0; c < 64; c += 32) {
                            float s[32];
                            tc::tmem_ld32(s_half + c, s);
                            tc::tmem_wait_ld();
                            const uint32_t see = live ? seen_bits(words, 2 * a.W, tok0 + 64 * half + c - x.len, x.rows, j) : 0u;
                            uint32_t hidden[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) hidden[i] = __float_as_uint(see & (1u << i) ? s[i] : -INFINITY);
                            tc::tmem_st32(s_half + c, hidden);
                        }
                        tc::tmem_wait_st();
                    }
                    if (!C::kHold && active) {
                        // 96 registers a thread (the warps that unpack need their share) and little code: 32 columns at
                        // a time, read from tensor memory for their maximum and again for their weights
                        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
                        for (int c = 0; c < 64; c += 32) {
                            float s[32];
                            tc::tmem_ld32(s_half + c, s);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i += 2) mx[(i >> 1) & 1] = max3(mx[(i >> 1) & 1], s[i], s[i + 1]);
                        }
                        const float top = fmaxf(mx[0], mx[1]) * scale;
                        const bool over = top > m + (kSlack + C::kLift);
                        if (__any_sync(0xffffffffu, over)) {
                            const float to = over ? top - C::kLift : m;
                            const float f = to == -INFINITY ? 1.f : ex2(m - to);
                            m = to;
                            l *= f;
                            if (u > 0 || half > 0) {  // else nothing is in O
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
                        }
                        const float ref = m == -INFINITY ? 0.f : m;
                        const float2 by = {scale, scale}, off = {-ref, -ref};
                        float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
                        for (int c = 0; c < 64; c += 32) {
                            float s[32];
                            uint32_t r[16];
                            tc::tmem_ld32(s_half + c, s);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 arg = fma2({s[2 * i], s[2 * i + 1]}, by, off);
                                const float2 e = {ex2(arg.x), ex2(arg.y)};
                                sum[i & 1] = add2(sum[i & 1], e);
                                r[i] = pack_half(e.x, e.y);
                            }
                            tc::tmem_st16(s_half + c / 2, r);  // over columns that were read
                        }
                        sum[0] = add2(sum[0], sum[1]);
                        l += sum[0].x + sum[0].y;
                        tc::tmem_wait_st();
                        tc::tc_fence_before();
                    }
                    if (C::kHold && active) {
                        float s[64];
                        tc::tmem_ld32(s_half, s);
                        tc::tmem_ld32(s_half + 32, s + 32);
                        tc::tmem_wait_ld();
                        if (!C::FOUR && tail) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                // lines beyond the unit's see nothing; what they hold is not read
                                const uint32_t see = live ? seen_bits(words, 2 * a.W, tok0 + 64 * half + 32 * c - x.len, x.rows, j) : 0u;
#pragma unroll
                                for (int i = 0; i < 32; ++i) s[32 * c + i] = see & (1u << i) ? s[32 * c + i] : -INFINITY;
                            }
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                        if (C::FOUR) {
#pragma unroll
                            for (int i = 0; i < 64; i += 2) mx[(i >> 1) & 1] = max3(mx[(i >> 1) & 1], s[i], s[i + 1]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 64; i += 4)
#pragma unroll
                                for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], s[i + c]);
                        }
                        const float top = (C::FOUR ? fmaxf(mx[0], mx[1]) : fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]))) * scale;
                        if (!C::FOUR && u == 0 && half == 0) {
                            m = top;
                        } else if (__any_sync(0xffffffffu, top > m + (kSlack + C::kLift))) {
                            const float to = top > m + (kSlack + C::kLift) ? top - C::kLift : m;
                            const float f = to == -INFINITY ? 1.f : ex2(m - to);
                            m = to;
                            l *= f;
                            if (!C::FOUR || u > 0 || half > 0) {  // else nothing is in O
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
                            r[i] = C::FOUR ? pack_half(e.x, e.y) : pack(e.x, e.y);
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
                // (values in 4 bits are multiplied as eighths of themselves)
                const float inv = (whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f) * (C::FOUR ? 8.f : 1.f);
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
                                    if constexpr (C::FOUR) {
                                        // infinite values are those of no numbers: 16 columns at a time
                                        const unsigned char *scales = static_cast<const unsigned char *>(a.v_cache) +
                                                                      ((size_t)pg * a.H + x.head) * cache4::page_bytes(a.page, a.D) +
                                                                      cache4::code_bytes(a.page, a.D) + (size_t)(tok % a.page) * (a.D / 16);
#pragma unroll
                                        for (int k = 0; k < 4; k += 2) {
                                            const int d = c + 8 * k;
                                            if (d >= a.D || scales[d / 16] != cache4::kNoNumbers) continue;
#pragma unroll
                                            for (int e = 0; e < 8; ++e)
                                                if (((e >> 1) & 1) == hf) o[4 * k + e] = NAN;
                                        }
                                        continue;
                                    }
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
            for (uint32_t k = 0; k < (uint32_t)kCopies; ++k)
                if ((mine >> k) & 1u) tc::mbar_wait_drain(&copied[(next - 1 - k) % kCopies], ((next - 1 - k) / kCopies) & 1u, a.err);
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

template <typename C>
cudaError_t launch_tc_as(const TcParams &tp, int grid, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                         cudaStream_t s) {
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    auto kern = tree_attention_tc<C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, C::kThreads, C::kSmem, s, q, k, v, tp);
}

// what the launches share: how the work is cut and weighed, the map of the queries; false
// where that has no map
inline bool tc_params(TcParams &tp, const Params &given, int grid, CUtensorMap *q) {
    tp.p = given;
    Params &p = tp.p;
    const dspark_tree_attention_args &a = p.a;
    tp.op_rows = 128 / p.G;
    tp.inv_group = (65536 + p.G - 1) / p.G;
    p.tile_log2 = kTileLog2;
    p.small_rows = tp.op_rows;
    p.small_places = div_by(kTilePlaces);
    p.large_places = div_by(p.block_rows > tp.op_rows ? kDualPlaces : kTilePlaces);
    p.page = div_by(a.page);
    p.ctas = div_by(grid);
    p.unit_cost = kUnitCost;
    tp.box = a.page & -a.page;
    if (tp.box > kTile) tp.box = kTile;
    const uint64_t dims[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.N};
    const uint64_t strides[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_row * 2};
    const uint32_t bx[3] = {64, (uint32_t)p.G, (uint32_t)tp.op_rows};
    return encode_bf16_map3(q, a.q, dims, strides, bx);
}

}  // namespace

}  // namespace attn
}  // namespace dspark
