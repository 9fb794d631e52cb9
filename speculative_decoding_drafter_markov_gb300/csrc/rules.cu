// rules.cu -- repetition penalties, biases and grammar masks on the target's
// logits, between the target's pass and the verification.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "target.h"
#include "tc.cuh"

namespace dspark {

namespace {

// One CTA takes one request, one slice of the vocabulary and a run of the
// request's rows.  Few entries of a vocabulary stand in a text or a bias list, so
// the work is split in two:
// * the grammar covers every entry of a row: 16-byte pieces with forbidden entries
//   at -inf (a piece that is forbidden whole is not read; in place, one that is
//   allowed whole is not touched);
// * the text is counted into a word per entry of the slice in shared memory, shared
//   by the rows, the entries that any other rule can touch are listed, and these
//   are computed for every row, a thread each.  Drafted tokens are marked in the
//   words; a row counts those that it continues.
// Each warp has a part of the slice to itself after the counting: a list of its own,
// and two places in shared memory through which the rows' parts go, a bulk copy in
// while the row before is worked on.  The listed entries are computed there (as
// 2-byte reads and writes of global memory they took as long as half of the copy)
// and the grammar on the way out; no warp waits for another.  In place there is
// no copy to join, and the listed entries are scattered.
// Bound by HBM: the logits' one read and one write.  The text is read once per
// slice, from L2, which is why a slice is large.  512 requests of up to 9 rows,
// V = 129280, bf16, texts of up to 8192 tokens: 236 us, 5.7 TB/s; without the texts
// 212 us.  (The CTAs of a request counting its text together, as a cluster of 2 / 4 / 8
// through each other's shared memory, moved in step and took 3 / 13 / 35 us more than
// each counting alone.)
constexpr int kRulesThreads = 256;
constexpr int kBiasList = 256;   // bias entries of a slice kept in shared memory,
constexpr int kDraftList = 128;  // drafted tokens too
constexpr int kSearch = 8;       // entries of both up to which they are searched for every row
constexpr int kMarked = 24;      // marked entries of a warp prepared for all rows
constexpr int kWarps = kRulesThreads / 32;
constexpr int kPart = 2048;      // bytes of a row that a warp stages: its part of a slice
constexpr int kSliceBytes = kPart * kWarps;

// An entry's word: said in the prompt, marked (in the bias list or drafted), how often
// in the output text.  16 bits serve texts of up to 16383 tokens; half the shared
// memory leaves bf16 four CTAs on an SM instead of three: 243 us instead of 293 for
// texts of up to 8192 tokens.
template <typename Word>
struct Entry;
template <>
struct Entry<uint16_t> {
    static constexpr uint32_t kPrompt = 1u << 15, kMark = 1u << 14, kCount = kMark - 1;
    using Listed = uint32_t;
    static __device__ __forceinline__ void add(uint16_t *words, unsigned at, uint32_t x) {
        atomicAdd(reinterpret_cast<uint32_t *>(words) + (at >> 1), x << (16 * (at & 1)));
    }
    static __device__ __forceinline__ void set(uint16_t *words, unsigned at, uint32_t x) {
        atomicOr(reinterpret_cast<uint32_t *>(words) + (at >> 1), x << (16 * (at & 1)));
    }
    static __device__ __forceinline__ Listed listed(uint32_t word, int place) { return word | (uint32_t)place << 16; }
    static __device__ __forceinline__ uint32_t word(Listed l) { return l & 0xffffu; }
    static __device__ __forceinline__ int place(Listed l) { return (int)(l >> 16); }
};
template <>
struct Entry<uint32_t> {
    static constexpr uint32_t kPrompt = 1u << 31, kMark = 1u << 30, kCount = kMark - 1;
    using Listed = uint2;
    static __device__ __forceinline__ void add(uint32_t *words, unsigned at, uint32_t x) { atomicAdd(words + at, x); }
    static __device__ __forceinline__ void set(uint32_t *words, unsigned at, uint32_t x) { atomicOr(words + at, x); }
    static __device__ __forceinline__ Listed listed(uint32_t word, int place) { return make_uint2(word, (uint32_t)place); }
    static __device__ __forceinline__ uint32_t word(Listed l) { return l.x; }
    static __device__ __forceinline__ int place(Listed l) { return (int)l.y; }
};
constexpr int kShortText = Entry<uint16_t>::kCount;

// What a marked entry looks through: the slice's bias entries in their order and its
// drafted tokens, in shared memory; or, when they are more than fit there, all of the
// request's in global memory.
struct Marks {
    const int *id;
    const float *val;   // biases
    const int *at;      // drafts: the row, or NULL: the place in the list is the row
    int n;
};

// The marked entries of a warp.  Where a request's rows fit 64 bits and an entry has one
// bias at most, bit i of `where` says that it is the token of row i (i > 0); else bit 0 is
// set, and it is searched for in every row.
template <typename Listed>
struct Marked {
    uint64_t where[kWarps][kMarked];
    Listed entry[kWarps][kMarked];
    float bias[kWarps][kMarked];
};

struct RowRules {
    float rep, inv_rep, freq, pres;
};

// c: occurrences in the output and on the row's path
__device__ __forceinline__ float penalised(float z, uint32_t c, bool prompt, const RowRules &k) {
    if (prompt || c) z *= z > 0.f ? k.inv_rep : k.rep;
    z = fmaf(-k.freq, (float)c, z);
    if (c) z -= k.pres;
    return z;
}

// a marked entry by search: how often it was drafted on the path of row j (mine: its
// mask words, NULL: a chain), and its biases
__device__ __forceinline__ float searched(float z, uint32_t c, bool prompt, int v, const RowRules k, const Marks bias, const Marks draft,
                                       const uint64_t *mine, int j) {
#pragma unroll 1
    for (int i = 0; i < draft.n; ++i) {
        if (draft.id[i] != v) continue;
        const int at = draft.at ? draft.at[i] : i;
        if (at > 0 && (mine ? (mine[at >> 6] >> (at & 63)) & 1 : at <= j)) ++c;
    }
    z = penalised(z, c, prompt, k);
#pragma unroll 1
    for (int i = 0; i < bias.n; ++i)
        if (bias.id[i] == v) z += bias.val[i];
    return z;
}

__device__ __forceinline__ void put(float *p, float z) { *p = z; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float z) { *p = __float2bfloat16_rn(z); }

// a 16-byte piece with the entries whose bit is clear at -inf; keep[i]: the two bits
// of i as masks of 16 bits each
__device__ __forceinline__ uint4 forbid(uint4 v, uint32_t ok, const uint32_t *, float) {
    const uint32_t inf = 0xff800000u;
    return make_uint4(ok & 1 ? v.x : inf, ok & 2 ? v.y : inf, ok & 4 ? v.z : inf, ok & 8 ? v.w : inf);
}
__device__ __forceinline__ uint4 forbid(uint4 v, uint32_t ok, const uint32_t *keep, __nv_bfloat16) {
    const uint32_t inf = 0xff80ff80u, m0 = keep[ok & 3], m1 = keep[(ok >> 2) & 3], m2 = keep[(ok >> 4) & 3], m3 = keep[ok >> 6];
    return make_uint4((v.x & m0) | (inf & ~m0), (v.y & m1) | (inf & ~m1), (v.z & m2) | (inf & ~m2), (v.w & m3) | (inf & ~m3));
}

// `bits` bits of a grammar row from entry v on (kAligned: in one word)
template <bool kAligned>
__device__ __forceinline__ uint32_t allowed(const uint32_t *allow, int v, int bits) {
    const int sh = v & 31;
    uint32_t x = allow[v >> 5] >> sh;
    if (!kAligned && sh + bits > 32) x |= allow[(v >> 5) + 1] << (32 - sh);
    return x & ((1u << bits) - 1);
}

// Waits for the copy of a warp's row k (of its run; `left` rows to come, itself among
// them).  A wait that runs out is reported and ends the warp's work: the rows left are
// unspecified, but its copies under way, of this row and the next, have landed.
__device__ __noinline__ bool row_landed(uint64_t *landed, int k, int left, volatile int *abort_flag, int32_t *err) {
    if (tc::mbar_wait(&landed[k & 1], (k >> 1) & 1, abort_flag, err)) return true;
    for (int i = k; i < k + min(left, 2); ++i) tc::mbar_wait_drain(&landed[i & 1], (i >> 1) & 1, err);
    return false;
}

// kAligned: every row of T and out starts on a 16-byte boundary; else vec: T and out
// lie alike to 16 bytes
template <typename T, typename Word, bool kAligned>
__global__ void __launch_bounds__(kRulesThreads, sizeof(Word) <= sizeof(T) ? 4 : 3) logit_rules_kernel(const dspark_logit_rules_args a, int slice, bool vec) {
    extern __shared__ __align__(128) unsigned char stage[];  // [warp][2][kPart], then the slice's words
    using W = Entry<Word>;
    Word *word = reinterpret_cast<Word *>(stage + 2 * kSliceBytes);
    __shared__ uint64_t landed[kWarps][2];
    __shared__ int abort_word;
    __shared__ int bias_id[kBiasList];
    __shared__ float bias_val[kBiasList];
    __shared__ int bias_n, draft_n;
    __shared__ int draft_id[kDraftList], draft_at[kDraftList];
    __shared__ Marked<typename Entry<Word>::Listed> marked;
    __shared__ uint32_t keep[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    after_predecessor();
    if (kAligned) vec = true;
    if (tid < 4) keep[tid] = (tid & 1 ? 0xffffu : 0u) | (tid & 2 ? 0xffff0000u : 0u);
    __syncthreads();
    const int r = blockIdx.y, v0 = blockIdx.x * slice, v1 = min(a.V, v0 + slice);
    // the request's numbers, all loads in flight together
    const int row0 = a.row_start[r], row_end = a.row_start[r + 1];
    RowRules k;
    k.rep = a.rep ? a.rep[r] : 1.f;
    k.freq = a.freq ? a.freq[r] : 0.f;
    k.pres = a.pres ? a.pres[r] : 0.f;
    int n = a.hist ? a.hist_len[r] : 0, np = a.hist && a.prompt_len ? a.prompt_len[r] : 0;
    int b0 = a.bias_start ? a.bias_start[r] : 0, b1 = a.bias_start ? a.bias_start[r + 1] : 0;
    if (row0 == row_end) return;
    const bool report = tid == 0 && blockIdx.x == 0 && blockIdx.z == 0;
    if (row0 < 0 || row_end < row0 || row_end > a.N || (a.mask && row_end - row0 > 64 * a.W)) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        return;
    }
    const int rows = row_end - row0;
    const int j0 = (int)((long long)rows * blockIdx.z / gridDim.z), j1 = (int)((long long)rows * (blockIdx.z + 1) / gridDim.z);
    if (n < 0 || n > a.max_hist || np < 0 || np > n) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        n = max(0, min(n, a.max_hist));
        np = max(0, min(np, n));
    }
    if (b0 < 0 || b1 < b0 || b1 > a.n_bias) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        b0 = b1 = 0;
    }
    if (j0 == j1) return;
    k.inv_rep = 1.f / k.rep;
    const bool penal = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
    const bool path = penal && a.tok;
    Marks bias{bias_id, bias_val, nullptr, 0}, draft{draft_id, nullptr, draft_at, 0};

    const int words = (a.V + 31) / 32;
    const bool in_place = a.T == a.out;
    auto grammar = [&](int row) -> const uint32_t * {
        const int m = a.allow ? a.allow_row[row] : -1;
        if (tid == 0 && m >= a.n_allow) set_err(a.err, DSPARK_ERR_RANGE);
        return m >= 0 && m < a.n_allow ? a.allow + (size_t)m * words : nullptr;
    };
    constexpr int E = 16 / (int)sizeof(T);
    constexpr uint32_t kAll = (1u << E) - 1;
    // the pieces [va, vb) of a row's entries [lo, hi) lie on 16-byte boundaries of memory;
    // what is left before and after them goes entry by entry
    auto pieces = [&](const T *src, int lo, int hi, int &va, int &vb) {
        if (kAligned) {
            va = lo;
            vb = hi;
            return;
        }
        va = vb = hi;
        if (!vec) return;
        const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(src + lo) & 15)) & 15) / (int)sizeof(T);
        va = min(hi, lo + lead);
        vb = va + (hi - va) / E * E;
    };
    auto copy_row = [&](int row) {
        const uint32_t *allow = grammar(row);
        const T *src = static_cast<const T *>(a.T) + (size_t)row * a.V;
        T *dst = static_cast<T *>(a.out) + (size_t)row * a.V;
        if (!in_place || allow) {
            constexpr int U = 4;
            int va, vb;
            pieces(src, v0, v1, va, vb);
            for (int first = va + E * tid; first < vb; first += U * E * kRulesThreads) {
                uint32_t ok[U];
                uint4 raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = first + u * E * kRulesThreads;
                    ok[u] = kAll;
                    if (allow && v < vb) ok[u] = allowed<kAligned>(allow, v, E);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = first + u * E * kRulesThreads;
                    raw[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (v < vb && ok[u] && !(in_place && ok[u] == kAll)) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(src + v));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = first + u * E * kRulesThreads;
                    if (v >= vb || (in_place && ok[u] == kAll)) continue;
                    if (allow) raw[u] = forbid(raw[u], ok[u], keep, T());
                    __stcs(reinterpret_cast<uint4 *>(dst + v), raw[u]);
                }
            }
            for (int i = tid; !kAligned && i < (va - v0) + (v1 - vb); i += kRulesThreads) {
                const int v = i < va - v0 ? v0 + i : vb + i - (va - v0);
                dst[v] = !allow || allowed<true>(allow, v, 1) ? src[v] : T(-INFINITY);
            }
        }
    };
    if (!penal && b1 == b0) {
        for (int j = j0; j < j1; ++j) copy_row(row0 + j);
        return;
    }

    // this warp's part of the slice
    const bool staged = vec && !in_place;
    const int part = slice / kWarps, lo = min(v1, v0 + warp * part), hi = min(v1, lo + part);
    unsigned char *places = stage + warp * 2 * kPart;
    auto load = [&](int j) {
        const T *src = static_cast<const T *>(a.T) + (size_t)(row0 + j) * a.V;
        int va, vb;
        pieces(src, lo, hi, va, vb);
        const int b = (j - j0) & 1;
        const uint32_t bytes = (uint32_t)(vb - va) * (uint32_t)sizeof(T);
        tc::mbar_expect_tx(&landed[warp][b], bytes);
        if (bytes) tc::bulk_load(places + b * kPart, src + va, bytes, &landed[warp][b]);
    };
    if (lane == 0) {
        tc::mbar_init(&landed[warp][0], 1);
        tc::mbar_init(&landed[warp][1], 1);
        tc::fence_mbar_init();
        if (staged) {
            load(j0);
            if (j0 + 1 < j1) load(j0 + 1);
        }
    }
    if (tid == 0) abort_word = bias_n = draft_n = 0;
    // the grammar's bits of a row are read a row ahead, the first during the counting
    constexpr int kMine = kPart / 16 / 32;  // a lane's pieces
    auto grammar_bits = [&](int j, uint32_t (&ok)[kMine]) {
        const uint32_t *allow = grammar(row0 + j);
        const T *src = static_cast<const T *>(a.T) + (size_t)(row0 + j) * a.V;
        int va, vb;
        pieces(src, lo, hi, va, vb);
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int v = va + E * (lane + 32 * u);
            ok[u] = allow && v < vb ? allowed<kAligned>(allow, v, E) : kAll;
        }
        return allow;
    };
    uint32_t ok[kMine];
    const uint32_t *allow = staged ? grammar_bits(j0, ok) : nullptr;
    // the first tokens of the text are on their way while the words are cleared
    // (16 bytes at a time between the row's first and last 16-byte boundary)
    constexpr int kAhead = 4;
    const int32_t *text = a.hist + (size_t)r * a.max_hist;
    if (!penal) n = 0;
    const int lead = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(text) & 15)) & 15) / 4), quads = (n - lead) / 4;
    const int4 *text4 = reinterpret_cast<const int4 *>(text + lead);
    int4 ahead[kAhead];
    auto quad = [&](int q) { return q < quads ? text4[q] : make_int4(0, 0, 0, 0); };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = quad(tid + i * kRulesThreads);
    constexpr int kWords16 = 16 / (int)sizeof(Word);
    for (int i = kWords16 * tid; i < slice; i += kWords16 * kRulesThreads)
        *reinterpret_cast<uint4 *>(word + i) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const unsigned width = v1 - v0;
    unsigned most = 0;  // largest token: those out of range are reported once
    auto count = [&](int i, int v) {
        most = max(most, (unsigned)v);
        const unsigned at = (unsigned)v - v0;
        if (at < width) {
            if (i < np) W::set(word, at, W::kPrompt);
            else W::add(word, at, 1u);
        }
    };
    auto count4 = [&](int q, const int4 &v) {
        const int i = lead + 4 * q;
        if (i >= np) {
            most = max(max(max(most, (unsigned)v.x), max((unsigned)v.y, (unsigned)v.z)), (unsigned)v.w);
            const unsigned x = (unsigned)v.x - v0, y = (unsigned)v.y - v0, z = (unsigned)v.z - v0, w = (unsigned)v.w - v0;
            if (x < width) W::add(word, x, 1u);
            if (y < width) W::add(word, y, 1u);
            if (z < width) W::add(word, z, 1u);
            if (w < width) W::add(word, w, 1u);
        } else {
            count(i, v.x);
            count(i + 1, v.y);
            count(i + 2, v.z);
            count(i + 3, v.w);
        }
    };
#pragma unroll 1
    for (int q = tid; q < quads; q += kRulesThreads) {
        const int4 v = ahead[0];
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
        ahead[kAhead - 1] = quad(q + kAhead * kRulesThreads);
        count4(q, v);
    }
    if (tid < lead) count(tid, text[tid]);
    if (tid < n - lead - 4 * quads) count(lead + 4 * quads + tid, text[lead + 4 * quads + tid]);
    if (most >= (unsigned)a.V) set_err(a.err, DSPARK_ERR_RANGE);
    if (path)  // whatever a row of the run may continue
        for (int at = 1 + tid; at < rows; at += kRulesThreads) {
            const int v = a.tok[row0 + at];
            if ((unsigned)v >= (unsigned)a.V) set_err(a.err, DSPARK_ERR_RANGE);
            if (v >= v0 && v < v1) {
                W::set(word, v - v0, W::kMark);
                const int i = atomicAdd(&draft_n, 1);
                if (i < kDraftList) {
                    draft_id[i] = v;
                    draft_at[i] = at;
                }
            }
        }
    if (b1 > b0 && tid < 32) {  // one warp, so that the list keeps the entries' order
        int found = 0;
        for (int i = b0; i < b1; i += 32) {
            const int v = i + lane < b1 ? a.bias_id[i + lane] : v0;
            if ((unsigned)v >= (unsigned)a.V) set_err(a.err, DSPARK_ERR_RANGE);
            const bool in = i + lane < b1 && v >= v0 && v < v1;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            const int at = found + __popc(who & ((1u << lane) - 1));
            if (in) {
                W::set(word, v - v0, W::kMark);
                if (at < kBiasList) {
                    bias_id[at] = v;
                    bias_val[at] = a.bias_val[i + lane];
                }
            }
            found += __popc(who);
        }
        if (lane == 0) bias_n = found;
    }
    __syncthreads();
    bias.n = bias_n;
    if (bias.n > kBiasList) bias = Marks{a.bias_id + b0, a.bias_val + b0, nullptr, b1 - b0};
    draft.n = draft_n;
    if (draft.n > kDraftList) draft = Marks{a.tok + row0, nullptr, nullptr, rows};
    // The warp's list of touched entries, over its words: a lane takes `part / 32` of
    // them into registers.  With more entries than fit there the words stay, and are
    // searched for every row.
    constexpr int kPacked = 4 / (int)sizeof(Word);  // words of a register
    constexpr int kLaneWords = kPart / (int)sizeof(T) / 32 / kPacked;
    Word *mine = word + warp * part;
    typename W::Listed *list = reinterpret_cast<typename W::Listed *>(word + warp * part);
    int listed = 0;
    {
        uint32_t w[kLaneWords];
        int n_own = 0;
#pragma unroll
        for (int i = 0; i < kLaneWords; ++i) {
            w[i] = 32 * i * kPacked < part ? reinterpret_cast<const uint32_t *>(mine)[32 * i + lane] : 0u;
            if (kPacked == 2) n_own += ((w[i] & 0xffffu) != 0) + ((w[i] >> 16) != 0);
            else n_own += w[i] != 0;
        }
        int at = n_own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += y;
        }
        listed = __shfl_sync(0xffffffffu, at, 31);
        at -= n_own;
        if (listed <= part / 2) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kLaneWords; ++i) {
                if (!w[i]) continue;
                const int place = (32 * i + lane) * kPacked;
                if (kPacked == 1) {
                    list[at++] = W::listed(w[i], place);
                } else {
                    if (w[i] & 0xffffu) list[at++] = W::listed(w[i] & 0xffffu, place);
                    if (w[i] >> 16) list[at++] = W::listed(w[i] >> 16, place + 1);
                }
            }
            __syncwarp();
        }
    }
    const bool by_list = listed <= part / 2;
    // The marked entries among them get a list of their own, of what they found in the lists
    // of biases and drafts (the warp looks for an entry together); where they stood is left
    // as if untouched.  (235 requests of up to 15 rows, V = 2656, texts of up to 855 tokens,
    // 64 biases: 29 us; with every marked entry searched for in every row 78 to 100.)
    int prepared = 0;
    if (bias.n + draft.n > kSearch) {
        const int n_all = by_list ? listed : part;
        for (int i0 = 0; i0 < n_all && prepared < kMarked; i0 += 32) {
            const int i = i0 + lane;
            uint32_t w = 0;
            if (i < n_all) w = by_list ? W::word(list[i]) : (uint32_t)mine[i];
            const uint32_t who = __ballot_sync(0xffffffffu, (w & W::kMark) != 0);
            const int at = prepared + __popc(who & ((1u << lane) - 1));
            if ((w & W::kMark) && at < kMarked) {
                const int place = by_list ? W::place(list[i]) : i;
                marked.entry[warp][at] = W::listed(w, place);
                if (by_list) list[i] = W::listed(0u, place);
                else mine[i] = 0;
            }
            prepared = min(kMarked, prepared + __popc(who));
        }
        __syncwarp();
        for (int e = 0; e < prepared; ++e) {
            const int v = lo + W::place(marked.entry[warp][e]);
            uint64_t where = rows > 64;  // bit 0: to be searched for in every row
            float val = 0.f;
            int found = 0;
            for (int i0 = 0; i0 < draft.n; i0 += 32) {
                const int i = i0 + lane;
                const bool hit = i < draft.n && draft.id[i] == v;
                if (hit) where |= 1ull << ((draft.at ? draft.at[i] : i) & 63);
            }
            for (int i0 = 0; i0 < bias.n; i0 += 32) {
                const int i = i0 + lane;
                const bool hit = i < bias.n && bias.id[i] == v;
                if (hit) val = bias.val[i];
                found += __popc(__ballot_sync(0xffffffffu, hit));
            }
            const uint32_t lo32 = __reduce_or_sync(0xffffffffu, (uint32_t)where), hi32 = __reduce_or_sync(0xffffffffu, (uint32_t)(where >> 32));
            const uint32_t bits = __reduce_or_sync(0xffffffffu, __float_as_uint(val));  // of one entry, if there is one
            if (lane == 0) {
                marked.where[warp][e] = (uint64_t)hi32 << 32 | lo32 | (found > 1);
                marked.bias[warp][e] = __uint_as_float(bits);
            }
        }
        __syncwarp();
    }
    // f(place in the part, word) for the touched entries, a lane each
    auto touched = [&](auto f) {
        if (by_list) {
            for (int i = lane; i < listed; i += 32) f(W::place(list[i]), W::word(list[i]));
        } else {
            for (int i = lane; i < part; i += 32)
                if (mine[i]) f(i, (uint32_t)mine[i]);
        }
    };

    // entry v of row j, whose word is w
    auto value = [&](int j, int v, uint32_t w, float z) {
        if (w & W::kMark)
            return searched(z, w & W::kCount, w & W::kPrompt, v, k, bias, draft, a.mask ? a.mask + (size_t)(row0 + j) * a.W : nullptr, j);
        return penalised(z, w & W::kCount, w & W::kPrompt, k);
    };
    auto scatter = [&](int j, int v, uint32_t w, const uint32_t *allow, const T *src, T *dst) {
        if (!allow || allowed<true>(allow, v, 1)) put(dst + v, value(j, v, w, to_f32(src[v])));
    };

    if (!staged) {
        for (int j = j0; j < j1; ++j) copy_row(row0 + j);
        __syncthreads();  // another thread's pieces are written
        for (int j = j0; j < j1; ++j) {
            const uint32_t *allow = grammar(row0 + j);
            const T *src = static_cast<const T *>(a.T) + (size_t)(row0 + j) * a.V;
            T *dst = static_cast<T *>(a.out) + (size_t)(row0 + j) * a.V;
            touched([&](int i, uint32_t w) { scatter(j, lo + i, w, allow, src, dst); });
            __syncwarp();
            if (lane < prepared) {
                const auto m = marked.entry[warp][lane];
                scatter(j, lo + W::place(m), W::word(m), allow, src, dst);
            }
        }
        return;
    }

    volatile int *abort_flag = &abort_word;
    for (int j = j0; j < j1; ++j) {
        const int b = (j - j0) & 1;
        uint32_t ok_next[kMine];
        const uint32_t *allow_next = j + 1 < j1 ? grammar_bits(j + 1, ok_next) : nullptr;
        const T *src = static_cast<const T *>(a.T) + (size_t)(row0 + j) * a.V;
        T *dst = static_cast<T *>(a.out) + (size_t)(row0 + j) * a.V;
        int va, vb;
        pieces(src, lo, hi, va, vb);
        T *row = reinterpret_cast<T *>(places + b * kPart) - va;  // entry v at row[v]
        for (int i = lane; !kAligned && i < (va - lo) + (hi - vb); i += 32) {
            const int v = i < va - lo ? lo + i : vb + i - (va - lo);
            dst[v] = !allow || allowed<true>(allow, v, 1) ? src[v] : T(-INFINITY);
        }
        int here = 1;
        if (lane == 0) here = tc::mbar_try_wait(&landed[warp][b], ((j - j0) >> 1) & 1) || row_landed(landed[warp], j - j0, j1 - j, abort_flag, a.err);
        if (!__shfl_sync(0xffffffffu, here, 0)) return;
        touched([&](int i, uint32_t w) {
            const int v = lo + i;
            if (!kAligned && (v < va || v >= vb)) scatter(j, v, w, allow, src, dst);
            else put(row + v, value(j, v, w, to_f32(row[v])));
        });
        if (prepared > 0) {
            __syncwarp();
            if (lane < prepared) {
                const auto m = marked.entry[warp][lane];
                const uint32_t w = W::word(m);
                const int v = lo + W::place(m);
                const uint64_t where = marked.where[warp][lane];
                if (!kAligned && (v < va || v >= vb)) {
                    scatter(j, v, w, allow, src, dst);
                } else {
                    float z = to_f32(row[v]);
                    if (where & 1) {
                        z = value(j, v, w, z);
                    } else {
                        const uint64_t seen = a.mask ? a.mask[(size_t)(row0 + j) * a.W] : j < 63 ? (2ull << j) - 1 : ~0ull;
                        z = penalised(z, (w & W::kCount) + __popcll(where & seen), w & W::kPrompt, k) + marked.bias[warp][lane];
                    }
                    put(row + v, z);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kMine; ++u) {
            const int v = va + E * (lane + 32 * u);
            if (v >= vb) break;
            uint4 q = *reinterpret_cast<const uint4 *>(row + v);
            if (ok[u] != kAll) q = forbid(q, ok[u], keep, T());
            __stcs(reinterpret_cast<uint4 *>(dst + v), q);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && j + 2 < j1) load(j + 2);
        allow = allow_next;
#pragma unroll
        for (int u = 0; u < kMine; ++u) ok[u] = ok_next[u];
    }
}

template <typename T, typename Word>
cudaError_t launch_as(const dspark_logit_rules_args &a, cudaStream_t s) {
    // The four CTAs that an SM holds: where requests are few their rows are spread, at the
    // price of counting the text for each run of rows; the slices are made smaller only
    // where even a CTA for every row leaves SMs empty.  (4 requests of up to 9 rows, V =
    // 129280, texts of up to 8192: 11.8 us, with small slices first 19.5; 16 requests: 18.8
    // and 32; up to 17 rows, texts of up to 1000, 4 requests: 9.4 and 25.)
    const long long want = 4ll * sm_count(), per = (a.N + a.R - 1) / a.R;
    int slice = kSliceBytes / (int)sizeof(T);
    while (slice > 1024 && a.R * per * ((a.V + slice - 1) / slice) < sm_count()) slice /= 2;
    const int slices = (a.V + slice - 1) / slice;
    // of one size, whole 64 entries for a warp
    slice = ((a.V + slices - 1) / slices + 64 * kWarps - 1) / (64 * kWarps) * (64 * kWarps);
    long long runs = (want + (long long)slices * a.R - 1) / ((long long)slices * a.R);
    if (runs > per) runs = per;
    if (runs < 1) runs = 1;
    const dim3 grid(slices, a.R, (unsigned)runs);
    const size_t smem = 2 * kSliceBytes + sizeof(Word) * (kSliceBytes / sizeof(T));
    const uintptr_t t = reinterpret_cast<uintptr_t>(a.T), o = reinterpret_cast<uintptr_t>(a.out);
    const bool aligned = ((t | o | (uintptr_t)a.V * sizeof(T)) & 15) == 0;
    auto kern = aligned ? logit_rules_kernel<T, Word, true> : logit_rules_kernel<T, Word, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, kRulesThreads, smem, s, a, slice, ((t ^ o) & 15) == 0);
}

}  // namespace

cudaError_t launch_logit_rules(const dspark_logit_rules_args &a, cudaStream_t s) {
    if (a.dtype != DSPARK_BF16) return launch_as<float, uint32_t>(a, s);
    return !a.hist || a.max_hist <= kShortText ? launch_as<__nv_bfloat16, uint16_t>(a, s) : launch_as<__nv_bfloat16, uint32_t>(a, s);
}

}  // namespace dspark
