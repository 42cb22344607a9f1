// Decoding attention over a paged key/value cache: Nq new query rows of each
// sequence against the rows its block table names, sequences of different
// lengths, pages in bf16 or in e4m3 with one scale per token and head.
//
// Every cached row is read once for the R = (H / Hkv) * Nq <= 32 query rows of
// its kv head, so the work is bound by HBM.  What the kernel has to do beside
// the loads is little, and is laid out so that it stays little in every type:
//   S_t^T = K_t Q^T      A = the tile's 128 keys, B = the query rows (N = 16 ..)
//   O^T  += V_t^T P_t^T  A = V read transposed (MN-major), B = P_t, O^T in TMEM
// With the keys on the MMA's M side a tile costs one read of K and V from
// shared memory (N is 16 to 64 columns), a softmax thread owns one key and up to
// sixteen rows' scores, nothing is computed for absent query rows past the next 1,
// 4, 8, 16 or 32, and no thread needs another's score: the running maximum m of a
// row (the reference) moves only when some key passes it by 2^kSlack (a vote of the
// four warps) or, in an e4m3 cache, at every 32nd tile, the row sums stay one partial per thread until the end, and the rescale of O^T
// touches few columns.  Neighbouring rows go through the fp32 units in pairs.
//
// e4m3 pages are multiplied as they are.  A bf16 query row, times the power of
// two that brings its largest entry into [2^7, 2^8), is a + b / 32 with e4m3
// numbers a and b (8 significant bits = 4 + 4; what a leaves is at most 8), exact
// where an entry is at least 2^-14 of the largest and off by at most 2^-22 of that
// below.  B holds the rows' first terms and, RP columns on, their second terms, and
// the two scores are added in fp32.  K's scale is the softmax thread's own
// (one thread, one key).  V's scale vs goes into P: w = 2^(x - m) vs kPScale with
// m the reference of x + log2 vs, so that w <= 448, as two e4m3 terms again, the
// second times 28 and with columns of O^T of its own.  These end at 2^-20.6 of the
// reference while the row sum counts every weight, so one early key must not set the
// reference of a long tail: every 32 tiles it is taken from the tile at hand, and O
// and the row sum, which are fp32, are scaled up to it.  A row of zeros has scale 0
// and weighs nothing.  No pass converts the pages, and shared memory sees each of
// their bytes twice.
//
// Work: the tiles of all (sequence, kv head) pairs, in order, are one list that
// the CTAs share evenly (List), found on the device from the lengths, so that
// ragged batches stay balanced and a captured graph replays with other lengths.
// A pair that one CTA holds whole is finished there.  The others leave O / l and
// LSE of their part in slot c + i (CTA c, pair i: along the list either c or i
// grows, so slots are unique), and the combine kernel joins a pair's slots in
// order.  A small call (short table, few pairs) takes no list and no second kernel:
// a cluster of CTAs shares a pair, and joins its parts through their shared memory.
//
// Warps: 0-3 (and 8-11) softmax, four warps for a group of query rows, which need
// nothing of one another; 4 loads K, 7 V, 5 issues MMAs, 6 lays out the queries
// of a pair and loads its scales.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kTile = 128;              // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kMinLogScale = -60.0f;  // V scales below 2^-60 no longer move the reference,
                                        // whose sum of weights would leave fp32's range
constexpr float kNoMax = -3.402823466e38f;   // running maximum of a row that has seen no key
constexpr int kSoftBar = 1;             // named barrier of softmax group 0
constexpr int kMaxCluster = 8;          // most CTAs that share a pair without a list

struct PagedParams {
    const __nv_bfloat16* q;             // rows i * R .. of pair i = b * Hkv + g
    const float* scales;
    const int* table;
    const int* seqlens;
    __nv_bfloat16* o;
    float* lse;
    float* part_o;                      // [slots][R][d]
    float* part_lse;                    // [slots][R], log2
    int B, Hkv, Nq, R, n_pages, ps_shift, max_pages, causal;
    int ctas;                           // of the split kernel; in clusters: of a pair
    float scale_log2;
    DeviceStatus* status;
};

// Sizes of one variant: head dimension, page type, groups of query rows, and how many
// rows a group works on (of at least eight; the others are zero).
template <int D, bool F8, int G, int W>
struct Cfg {
    static constexpr int kRows = W > 8 ? W : 8;    // of Q, S and P that a softmax group owns
    static constexpr int RP = kRows * G;
    static constexpr int kThreads = 128 + 128 * G;
    static constexpr int kN = F8 ? 2 * RP : (RP < 16 ? 16 : RP);   // columns of S, rows of Q
    // P enters as the sum of two terms of its type, so that its rounding does not
    // show beside the output's (with one bf16 term the output's error was 1.4
    // times its rounding).
    static constexpr int kNP = 2 * RP;                             // columns of O, rows of P
    static constexpr int kRowBytes = F8 ? D : 2 * D;
    static constexpr int kSw = kRowBytes < 128 ? 64 : 128;         // swizzle = chunk width
    static constexpr int kChunks = kRowBytes / kSw;
    static constexpr int kTileBytes = kTile * kRowBytes;
    static constexpr int kQBytes = kN * kRowBytes;
    static constexpr int kPRow = F8 ? kTile : 2 * kTile;
    static constexpr int kPBytes = kNP * kPRow;
    static constexpr int kPBufs = !F8 && D == 128 && RP == 32 ? 1 : 2;   // no room for two there
    static constexpr int kScaleBytes = F8 ? 2 * kTile * 4 : 0;
    // bf16 rows of 128 fill an SM with one CTA.  Smaller ones leave less time a
    // tile, and with up to 8 rows two CTAs fit, so that one's softmax and
    // epilogue hide behind the other's.
    static constexpr int kCtas = kRowBytes <= 128 && RP == 8 ? 2 : 1;
    static constexpr int kStatic = F8 ? 2304 : 2048;   // shared memory beside the tiles
    static constexpr int kRing = (kCtas == 2 ? 113 : 227) * 1024 - 1024 - kStatic - 2 * kQBytes -
                                 kPBufs * kPBytes;
    static constexpr int kStages = kRing / (2 * kTileBytes + kScaleBytes);
    // Tiles of K, and of V, in flight at once: about 112 KB an SM.  More of them
    // slow the memory down: with all three stages in flight bf16 at d = 64 took
    // 84.1 us instead of 80.0 (B16 H16, 8192 keys), at d = 128 155.5 instead of 153.2
    // (B8 Hkv8, 32768 keys).  Rows of 64 bytes are bound by the number of copies
    // instead (103 us with this limit, 96 without: B16 H16, 16384 keys, pages of 16).
    static constexpr int kAhead =
        kRowBytes >= 128 ? (56 * 1024 / kCtas + kTileBytes / 2) / kTileBytes : kStages;
    static constexpr int kSmem =
        kStages * (2 * kTileBytes + kScaleBytes) + 2 * kQBytes + kPBufs * kPBytes + 1024;
    static constexpr int kCols = 2 * kN + kNP;
    static constexpr int kTmemCols = kCols <= 64 ? 64 : (kCols <= 128 ? 128 : 256);
    // Most tiles of a CTA where clusters share the pairs.  One sequence of 8 kv
    // heads, with clusters (of eight) and with the list: 1000 keys 5.4 and 6.4 us,
    // 2000 5.9 and 6.8; 4000 keys (four tiles a CTA) 7.9 and 7.6 in bf16 at d = 128,
    // 7.1 and 8.4 in e4m3, 7.0 and 7.6 at d = 64; 8000 keys 9.2 and 7.8 at d = 64.
    static constexpr int kClusterTiles = kRowBytes <= 128 ? 4 : 2;
    // How far a score may pass the reference before O is rescaled (log2): bf16 P
    // keeps its precision at any magnitude; e4m3 P ends at 448.
    static constexpr float kSlack = F8 ? 3.0f : 8.0f;
    static constexpr float kPScale = F8 ? 56.0f : 1.0f;            // 2^kSlack * kPScale = 448
    // The second term of an e4m3 query is stored times this.
    static constexpr float kQTerm2 = 32.0f;
    // e4m3's second term of P is stored times this, and its columns of O count that
    // much less: what a first term of up to 448 leaves is at most 16.
    static constexpr float kTerm2 = F8 ? kE4m3Term2 : 1.0f;
    // Every kRefTiles tiles e4m3's reference is taken anew, and may fall, but not by
    // more than kRefDrop (log2) below the largest so far.  A term's last half step is
    // 2^-10 / 28, so weights end at 2^-10 / 28 / 56 = 2^-20.6 of the reference: of the
    // 4096 keys that share one, at most 2^-8.6 of the largest product is lost, however
    // long the cache.  (With one reference for a whole pair, 4096 keys a stretch turn
    // into n.)  Four tokens a sequence, B8, 8 kv heads, 8K to 16K keys, without this,
    // every 32 and every 16 tiles: 16 rows of d = 128 40.8, 41.1 and 41.3 us, 32 rows
    // 52.6, 54.6 and 55.7; 16 rows of d = 64 36.0, 37.4 and 38.0; 8 rows alike.
    static constexpr int kRefTiles = F8 ? 32 : 0;
    static constexpr float kRefDrop = 24.0f;
};

__device__ __forceinline__ int clamped_len(const PagedParams& p, int b) {
    return min(max(p.seqlens[b], 0), p.max_pages << p.ps_shift);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// The list and how it is shared, as a warp sees it.  A pair counts its tiles and
// `extra` units more (its queries, first maximum and epilogue; none where there is
// a CTA for every tile); of the V units in all, CTA c holds c * size .. (c + 1) *
// size - 1.  No CTA between two others is empty, so the CTAs of a pair are
// neighbours.  Lane l knows the units of ceil(B / 32) neighbouring sequences b0 ..
// b1 - 1, which begin at unit `at` and end at `upto`.
struct List {
    int b0, b1, at, upto, V, size, extra;
    __device__ __forceinline__ List(const PagedParams& p, int lane) {
        const int per = (p.B + 31) / 32;
        b0 = min(p.B, lane * per);
        b1 = min(p.B, b0 + per);
        int tiles = 0, seqs = 0;
#pragma unroll 2
        for (int b = b0; b < b1; ++b) {
            const int t = tiles_of(clamped_len(p, b));
            tiles += t;
            seqs += t > 0;
        }
        extra = __reduce_add_sync(0xffffffffu, tiles) * p.Hkv > p.ctas;
        const int mine = (tiles + extra * seqs) * p.Hkv;
        upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        at = upto - mine;
        V = __shfl_sync(0xffffffffu, upto, 31);
        size = max(1, (int)((unsigned)(V + p.ctas - 1) / (unsigned)p.ctas));
    }
    // units of one sequence: all its kv heads
    __device__ __forceinline__ int units_of(const PagedParams& p, int len) const {
        return len > 0 ? (tiles_of(len) + extra) * p.Hkv : 0;
    }
    __device__ __forceinline__ int begin(int c) const { return min(V, c * size); }
    __device__ __forceinline__ int cta_of(int u) const {
        return (int)((unsigned)u / (unsigned)size);
    }
};

// A CTA's place in the list: pair (b, g), tile t of it, and the units left.
struct Cursor {
    int b, g, len, t, left, extra;
    // The place of CTA c, found by a warp together.
    __device__ __forceinline__ Cursor(const PagedParams& p, const List& list, int c) {
        const int begin = list.begin(c);
        b = g = len = t = 0;
        extra = list.extra;
        left = list.begin(c + 1) - begin;
        if (left <= 0) return;
        const bool here = list.at <= begin && begin < list.upto;
        const int owner = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        if (owner < 0) {                // (lengths that somebody changes under the kernel)
            left = 0;
            return;
        }
        if (here) {
            int at = list.at;
#pragma unroll 1
            for (b = list.b0; b < list.b1; ++b) {
                len = clamped_len(p, b);
                const int u = list.units_of(p, len);
                if (begin < at + u) break;
                at += u;
            }
            const int per = tiles_of(len) + extra;
            g = (begin - at) / per;
            t = (begin - at) - g * per - extra;        // -1: the pair's extra unit
        }
        b = __shfl_sync(0xffffffffu, b, owner);
        g = __shfl_sync(0xffffffffu, g, owner);
        t = __shfl_sync(0xffffffffu, t, owner);
        len = __shfl_sync(0xffffffffu, len, owner);
        if (b >= p.B || g < 0 || g >= p.Hkv || t >= tiles_of(len)) left = 0;
        if (t < 0) {
            left += t;
            t = 0;
        }
    }
    // Without a list: CTA `rank` of the `ctas` that share a pair.
    __device__ __forceinline__ Cursor(const PagedParams& p, int pair, int rank) {
        b = pair / p.Hkv;
        g = pair - b * p.Hkv;
        extra = 0;
        len = clamped_len(p, b);
        const int tiles = tiles_of(len), per = (tiles + p.ctas - 1) / p.ctas;
        t = rank * per;
        left = max(0, min(per, tiles - t));
    }
    // tiles of the current pair that belong to this CTA
    __device__ __forceinline__ int run() const { return min(tiles_of(len) - t, left); }
    // past `n` tiles of the current pair
    __device__ __forceinline__ void skip(const PagedParams& p, int n) {
        left -= n;
        t += n;
        if (left <= 0 || t < tiles_of(len)) return;
        t = 0;
        if ((left -= extra) <= 0) return;
        if (++g < p.Hkv) return;
        g = 0;
        do {                            // left > 0: a sequence with keys follows
            if (++b >= p.B) {
                left = 0;
                return;
            }
            len = clamped_len(p, b);
        } while (len == 0);
    }
};

// The library's bounded wait with only the first poll inlined.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int site, const WaitCtx& wc) {
    return fa_wait(bar, parity, site, wc);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int site, const WaitCtx& wc) {
    return mbar_try_wait(smem_u32(bar), parity) || wait_on(bar, parity, site, wc);
}
// Two barriers' phases, both tried before either answer is needed (16 rows of e4m3,
// d = 64: 37.5 us instead of 38.6 with one after the other).
__device__ __forceinline__ bool wait_both(uint64_t* a, uint64_t* b, uint32_t parity, int site,
                                          const WaitCtx& wc) {
    const bool there = mbar_try_wait(smem_u32(a), parity);
    const bool too = mbar_try_wait(smem_u32(b), parity);
    return (there && too) ||
           (wait_on(a, parity, site, wc) && wait_on(b, parity, site + 1, wc));
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int site,
                                          const WaitCtx& wc) {
    // a vote before the branch keeps the warp together where the phase is complete
    if (__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) return true;
    return __all_sync(0xffffffffu, wait_on(bar, parity, site, wc));
}

// Monotone map of a float's order onto signed integers (its own inverse).
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
}

// Rows r and r + 1 of a thread's W as a pair (with one row: and zero).
template <int W>
__device__ __forceinline__ uint64_t pair(const float (&x)[W], int r) {
    return f2(x[r], W > 1 ? x[(r + 1) % W] : 0.0f);
}
template <int W>
__device__ __forceinline__ uint64_t pair(const uint32_t (&x)[W], int r) {
    return f2(__uint_as_float(x[r]), W > 1 ? __uint_as_float(x[(r + 1) % W]) : 0.0f);
}
template <int W>
__device__ __forceinline__ void put(float (&x)[W], int r, uint64_t v) {
    float hi;
    f2_split(v, x[r], hi);
    if (W > 1) x[(r + 1) % W] = hi;
}

// m + log2 l for l > 0.  The exponent of l is added to m first: the two cancel
// where V's scales are small, and lg2.approx is off by 2^-22 absolutely only on
// [1, 2).
__device__ __forceinline__ float add_log2(float m, float l) {
    const int i = __float_as_int(l), e = (i >> 23) - 127;
    if (e == 128) return m + l;                   // infinity or NaN
    return (m + (float)e) + lg2(__int_as_float((i & 0x7fffff) | 0x3f800000));
}

// Sums v[r] over the warp, all rows at once: halving exchanges leave each lane
// with one row's total (RP = 32), or 32 / RP lanes with the same row's.
// Returns the total; `row` is the lane's row.
template <int RP>
__device__ __forceinline__ float warp_row_sums(float (&v)[RP], int lane, int& row) {
    row = 0;
    int w = RP;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (w > 1) {
            w >>= 1;
            const bool up = lane & off;
            if (up) row += w;
#pragma unroll
            for (int i = 0; i < RP / 2; ++i)
                if (i < w) {
                    const float give = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
    return v[0];
}

template <int D, bool F8, int G, int W, bool CLUSTER>
__global__ void __launch_bounds__((Cfg<D, F8, G, W>::kThreads), (Cfg<D, F8, G, W>::kCtas))
fa_decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedParams p) {
    using C = Cfg<D, F8, G, W>;
    constexpr int S = C::kStages, N = C::kN, NP = C::kNP, TB = C::kTileBytes, RP = C::RP;
    constexpr uint32_t kColO = 2 * N;             // S buffers at 0 and N
    extern __shared__ uint8_t dsm_raw[];
    // 32-bit shared addresses, 1024-byte aligned.  Stage s: V, then K.  At d = 64
    // the MMA's 128 rows reach past V's 64 columns: its second half reads K, into
    // rows of O^T that nobody reads.
    const uint32_t sKV = (smem_u32(dsm_raw) + 1023) & ~1023u;
    const uint32_t sQ = sKV + S * 2 * TB;         // [2]
    const uint32_t sP = sQ + 2 * C::kQBytes;      // [kPBufs]
    const uint32_t sScale = sP + C::kPBufs * C::kPBytes;  // [S][K, V][128] fp32
    // per stage: K, V and e4m3's scales are there; S and P V of the stage's tile are
    // complete, which also frees its K, and its V and scales
    __shared__ uint64_t bar_k[S], bar_v[S], bar_x[S], bar_s[S], bar_pv[S];
    __shared__ uint64_t bar_q[2], bar_q_free[2], bar_p[2], bar_drain;   // by pair; P by tile
    __shared__ float4 row_max[RP], row_sum[RP];   // a value a softmax warp
    __shared__ float q_scale[2][RP];              // e4m3: score of one code product, log2 units
    __shared__ int row_query[RP];                 // r % Nq
    // e4m3: a row's largest reference before the last time that it could fall (by
    // turns: one is read while the other is written)
    __shared__ float row_top[2][RP];
    __shared__ float cta_lse[RP];                 // in clusters: of this CTA's part, log2
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    const WaitCtx wc{p.status, &abort_sh}, dc{p.status, nullptr};   // dc: for drains
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            abort_sh = 0;
            for (int x = 0; x < 2; ++x) {
                mbar_init(&bar_q[x], 32);
                mbar_init(&bar_q_free[x], F8 ? 1 + 4 * G : 1);   // the last S MMA; scales read
                mbar_init(&bar_p[x], 128 * G);
            }
#pragma unroll 1
            for (int s = 0; s < S; ++s) {
                mbar_init(&bar_k[s], 1);
                mbar_init(&bar_v[s], 1);
                mbar_init(&bar_x[s], 32);
                mbar_init(&bar_s[s], 1);
                mbar_init(&bar_pv[s], 1);
            }
            mbar_init(&bar_drain, 1);
            fence_mbar_init();
        }
    } else if (warp == 5) {
        tmem_alloc(&tmem_base_sh, C::kTmemCols);
        tmem_relinquish();
    } else {
        // Query rows past R and columns of P past RP stay zero.
        const int x0 = (warp < 4 ? warp : warp - 2) * 32 + lane;
#pragma unroll 1
        for (int e = x0; e < (2 * C::kQBytes + C::kPBufs * C::kPBytes) / 16; e += C::kThreads - 64)
            sts_v4(sQ + e * 16, make_uint4(0u, 0u, 0u, 0u));
        if (warp == 6)
#pragma unroll 1
            for (int r = lane; r < RP; r += 32) {
                row_query[r] = r % p.Nq;
                cta_lse[r] = -CUDART_INF_F;       // a CTA without tiles
            }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    // Up to here nothing is read that an earlier kernel may have written: it may
    // still run.  Loads from here on are not ld.global.nc, whose data has to be
    // constant from the launch on.  The combine kernel may come in only now: it
    // reads the lengths before it waits for this one.
    pdl_wait();
    pdl_launch_dependents();
    // CTA c of the list; in clusters pair c
    const int c = CLUSTER ? blockIdx.x / p.ctas : blockIdx.x;
    Cursor cur = CLUSTER ? Cursor(p, c, cluster_rank()) : Cursor(p, List(p, lane), c);

    const int seg_shift = min(p.ps_shift, 7), seg = 1 << seg_shift;
    const int n_seg = kTile >> seg_shift, page_mask = (1 << p.ps_shift) - 1;
    // The page of lane's segment of the cursor's tile (0 where there is none).
    auto page_of = [&](const Cursor& at) {
        const int key = at.t * kTile + lane * seg;
        return (at.left > 0 && lane < n_seg && key < at.len)
                   ? p.table[(long long)at.b * p.max_pages + (key >> p.ps_shift)]
                   : 0;
    };

    if (warp == 4 || warp == 7) {
        // ------------------------------------------------------- loads
        // Boxes of up to 128 keys of one page.  Lane i holds segment i's place
        // in the pool; one elected lane issues, because a copy takes uniform
        // registers.
        const bool is_v = warp == 7;
        const CUtensorMap* map = is_v ? &tm_v : &tm_k;
        uint64_t* full = is_v ? bar_v : bar_k;
        uint64_t* empty = is_v ? bar_pv : bar_s;
        const int seg_bytes = seg * C::kSw;
        const uint64_t policy = l2_evict_first();
        const bool leader = elect_one();
        const int outside = p.n_pages * p.Hkv;
        bool ok = true;
        int gt = 0;                               // tiles loaded so far
        int page = page_of(cur);
#pragma unroll 1
        while (ok && cur.left > 0) {
            const Cursor at = cur;
            cur.skip(p, 1);
            const int page_next = page_of(cur);              // in flight during the wait
            const int s = gt % S;
            const int have = min(n_seg, (at.len - at.t * kTile + seg - 1) >> seg_shift);
            const bool known = (unsigned)page < (unsigned)p.n_pages;
            // a page outside the pool reads as zeros (past the map's last row)
            const int outer = known ? page * p.Hkv + at.g : outside;
            const int row = (at.t * kTile) & page_mask;      // of a page of 256; else 0
            if (gt >= S)
                ok = wait_warp(&empty[s], ((gt / S) - 1) & 1, is_v ? 101 : 100, wc);
            if (C::kAhead < S && gt >= C::kAhead)
                ok = ok &&
                     wait_warp(&full[(gt - C::kAhead) % S], ((gt - C::kAhead) / S) & 1, 103, wc);
            if (!ok) break;
            const uint32_t stage = sKV + s * 2 * TB + (is_v ? 0 : TB);
            if (leader) mbar_arrive_expect_tx(&full[s], have * seg_bytes * C::kChunks);
            __syncwarp();
#pragma unroll 2
            for (int i = 0; i < have; ++i) {
                const int at_row = __shfl_sync(0xffffffffu, outer, i);
                if (leader) {
#pragma unroll
                    for (int h = 0; h < C::kChunks; ++h)
                        tma_load_3d_at(stage + h * (kTile * C::kSw) + i * seg_bytes, map, &full[s],
                                       h * (F8 ? C::kSw : C::kSw / 2), row, at_row, policy);
                }
            }
            ++gt;
            page = page_next;
        }
        // No copy may still be on its way when the CTA ends, whatever the other
        // warps did.
#pragma unroll 1
        for (int t = max(0, gt - S); t < gt; ++t) wait(&full[t % S], (t / S) & 1, 102, dc);
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------- MMAs
        constexpr uint32_t idesc_s =
            F8 ? idesc_e4m3_f32(128, N) : idesc_bf16_f32(128, N, false, false);
        constexpr uint32_t idesc_o =
            F8 ? idesc_e4m3_f32(128, NP, true) : idesc_bf16_f32(128, NP, true, false);
        constexpr uint32_t kGroup = 8 * C::kSw;                      // 8 rows of a chunk
        auto desc = [&](uint32_t a, uint32_t lbo) {
            return C::kSw == 128 ? sdesc_sw128(a, lbo, kGroup) : sdesc_sw64(a, lbo, kGroup);
        };
        // The warp stays together and one elected lane issues, by a predicate:
        // descriptors then travel in uniform registers (a branch on lane == 0 cost
        // 12 us of 49 with 16 rows an e4m3 cache: B8, four tokens, 8K to 16K keys).
        // A second warp for P V, so that S never queues behind it, gave nothing
        // (41.2 and 40.8 us there) and takes registers (8 rows: 37.4 and 39.2).
        const bool leader = elect_one();
        // O^T (+)= V_u^T P_u^T
        auto pv = [&](int u, bool first) -> bool {
            const int s = u % S;
            if (!wait_warp(&bar_p[u & 1], (u >> 1) & 1, 104, wc) ||
                !wait_warp(&bar_v[s], (u / S) & 1, 105, wc))
                return false;
            tc_fence_after();
            // V transposed: 32 (e4m3) or 16 keys a step; the next chunk of
            // columns (d = 64: K) is the leading-dimension stride
            const uint64_t vd = desc(sKV + s * 2 * TB, C::kChunks == 2 ? kTile * C::kSw : TB);
            const uint64_t pd = sdesc_sw128(sP + u % C::kPBufs * C::kPBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < (F8 ? 4 : 8); ++kk) {
                const uint64_t a = vd + (uint64_t)(kk * (F8 ? 32 : 16) * C::kSw >> 4);
                const uint64_t b = pd + kmajor_step(kk, NP * 128);
                if (F8) mma_ss_f8_if(leader, tmem + kColO, a, b, idesc_o, !first || kk > 0);
                else mma_ss_if(leader, tmem + kColO, a, b, idesc_o, !first || kk > 0);
            }
            mma_commit_if(leader, &bar_pv[s]);
            return true;
        };
        bool ok = true;
        int gt = 0, pairs = 0;
        bool behind = false, first = false;   // P V of tile gt - 1 to come; it begins its pair
        for (; ok && cur.left > 0; ++pairs) {
            const int tiles = cur.run();
            cur.skip(p, tiles);
            // after the last pair: its last P V
            const int flush = cur.left <= 0;
            ok = wait_warp(&bar_q[pairs & 1], (pairs >> 1) & 1, 106, wc);
            tc_fence_after();
            const uint64_t qd = desc(sQ + (pairs & 1) * C::kQBytes, 16);
#pragma unroll 1
            for (int t = 0; ok && t < tiles + flush; ++t) {
                const int u = gt + t, s = u % S;
                if (t < tiles) {
                    if (!(ok = wait_warp(&bar_k[s], (u / S) & 1, 107, wc))) break;
                    tc_fence_after();
                    // S_u's buffer was read before P_{u-2} was complete
                    const uint64_t kd = desc(sKV + s * 2 * TB + TB, 16);
#pragma unroll
                    for (int kk = 0; kk < C::kRowBytes / 32; ++kk) {
                        const uint64_t a = kd + kmajor_step(kk, kTile * 128);
                        const uint64_t b = qd + kmajor_step(kk, N * 128);
                        if (F8) mma_ss_f8_if(leader, tmem + (u & 1) * N, a, b, idesc_s, kk > 0);
                        else mma_ss_if(leader, tmem + (u & 1) * N, a, b, idesc_s, kk > 0);
                    }
                    mma_commit_if(leader, &bar_s[s]);
                    mma_commit_if(leader && t + 1 == tiles, &bar_q_free[pairs & 1]);
                }
                // P V one tile behind, across pairs: the softmax warps have read
                // a pair's O before they give the next pair's first P
                if (behind) ok = pv(u - 1, first);
                behind = true;
                first = t == 0;
            }
            gt += tiles;
        }
        if (leader && !ok) {   // no MMA of this thread may still write TMEM at teardown
            mma_commit(&bar_drain);
            wait(&bar_drain, 0, 108, dc);
        }
        __syncwarp();
    } else if (warp == 6) {
        // ---------------------------------- query rows, and e4m3's scales
        bool ok = true;
        int pairs = 0;
        int gt = 0;                               // tiles whose scales are loaded
        while (cur.left > 0) {
            if (pairs >= 2)
                ok = wait_warp(&bar_q_free[pairs & 1], ((pairs >> 1) - 1) & 1, 109, wc);
            if (!ok) break;
            const uint32_t dst = sQ + (pairs & 1) * C::kQBytes;
            const __nv_bfloat16* src = p.q + ((long long)cur.b * p.Hkv + cur.g) * p.R * D;
            if constexpr (F8) {
                // eight lanes a row, D / 8 neighbouring entries each
                constexpr int E = D / 8;
                const int at = lane & 7;
#pragma unroll 1
                for (int r0 = 0; r0 < p.R; r0 += 4) {
                    const int r = r0 + (lane >> 3);
                    uint4 w[E / 8];
                    float x[E];
                    uint32_t amax = 0, c1[E / 4], c2[E / 4];
#pragma unroll
                    for (int e = 0; e < E / 8; ++e) {
                        w[e] = make_uint4(0u, 0u, 0u, 0u);
                        if (r < p.R)
                            w[e] = reinterpret_cast<const uint4*>(src + r * D + at * E)[e];
                        const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[8 * e + 2 * i] = __uint_as_float(u[i] << 16);
                            x[8 * e + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
                        }
                    }
                    // magnitudes order like their bits; a NaN only shifts the scale
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        amax = max(amax, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
                    for (int off = 4; off > 0; off >>= 1)
                        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, off));
                    // 2^k amax in [2^7, 2^8); k <= 120 (smaller rows keep fewer bits)
                    const int ex = (int)(amax >> 23) - 127;
                    const int k = min(7 - ex, 120);
                    const float up = __uint_as_float((uint32_t)(127 + k) << 23);
#pragma unroll
                    for (int e = 0; e < E; e += 4) {
                        float v[4];
                        c1[e / 4] = pack_e4m3x4(x[e] * up, x[e + 1] * up, x[e + 2] * up,
                                                x[e + 3] * up);
                        unpack_e4m3x4(c1[e / 4], v);
                        // (x up - v) kQTerm2; all of it exact
                        const float up2 = up * C::kQTerm2;
                        c2[e / 4] = pack_e4m3x4(fmaf(x[e], up2, -C::kQTerm2 * v[0]),
                                                fmaf(x[e + 1], up2, -C::kQTerm2 * v[1]),
                                                fmaf(x[e + 2], up2, -C::kQTerm2 * v[2]),
                                                fmaf(x[e + 3], up2, -C::kQTerm2 * v[3]));
                    }
                    if (r < p.R) {
                        if constexpr (E == 16) {       // one 16-byte unit, swizzled by r & 7
                            const uint32_t to = dst + r * 128 + ((at ^ (r & 7)) << 4);
                            sts_v4(to, make_uint4(c1[0], c1[1], c1[2], c1[3]));
                            sts_v4(to + RP * 128, make_uint4(c2[0], c2[1], c2[2], c2[3]));
                        } else {                       // half of one, swizzled by r / 2 & 3
                            const uint32_t to =
                                dst + r * 64 + (((at >> 1) ^ ((r >> 1) & 3)) << 4) + (at & 1) * 8;
                            sts_v2(to, c1[0], c1[1]);
                            sts_v2(to + RP * 64, c2[0], c2[1]);
                        }
                    }
                    // an infinite entry would saturate: the whole row becomes NaN
                    if (at == 0 && r < RP)
                        q_scale[pairs & 1][r] =
                            ex == 128 ? CUDART_NAN_F
                                      : p.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23);
                }
#pragma unroll 1
                for (int r = (p.R + 3) / 4 * 4 + lane; r < RP; r += 32)
                    q_scale[pairs & 1][r] = 0.0f;
            } else {
                constexpr int U = D / 8;      // 16-byte units of a row
#pragma unroll 2
                for (int e = lane; e < p.R * U; e += 32) {
                    const int r = e / U, u = e % U;
                    const uint4 w = reinterpret_cast<const uint4*>(src)[e];
                    sts_v4(dst + (u >> 3) * (N * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4), w);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar_q[pairs & 1]);
            ++pairs;
            if constexpr (F8) {
                // 128 keys' scales a tile, four bytes a lane and copy
                int page = page_of(cur);
#pragma unroll 1
                for (int t = cur.run(); ok && t > 0; --t, ++gt) {
                    const Cursor at = cur;
                    cur.skip(p, 1);
                    const int page_next = page_of(cur);
                    const int s = gt % S;
                    if ((unsigned)page >= (unsigned)p.n_pages) page = 0;
                    if (gt >= S) ok = wait_warp(&bar_pv[s], ((gt / S) - 1) & 1, 116, wc);
                    const uint32_t dst = sScale + s * C::kScaleBytes + lane * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = 32 * i + lane;
                        const int pg = __shfl_sync(0xffffffffu, page, j >> seg_shift);
                        const float* src = p.scales +
                                           (((long long)pg * p.Hkv + at.g) << (p.ps_shift + 1)) +
                                           ((at.t * kTile + j) & page_mask);
                        cp_async4(dst + 128 * i, src);
                        cp_async4(dst + kTile * 4 + 128 * i, src + (1 << p.ps_shift));
                    }
                    cp_async_arrive(&bar_x[s]);
                    page = page_next;
                }
            } else {
                cur.skip(p, cur.run());
            }
        }
        if (F8) cp_async_wait_all();
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax
        // Thread j of a group holds key j of the tile and the group's first W
        // rows.  A wait that gives up clears `ok` and skips the later waits, but
        // every thread stays in step with the named barriers.
        const int group = warp < 4 ? 0 : (warp >> 2) - 1, r0 = group * C::kRows;
        const int quarter = warp & 3, j = quarter * 32 + lane;
        const int bar_id = kSoftBar + group;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16) + r0;
        const uint32_t max_w = smem_u32(row_max + r0) + quarter * 4;   // this warp's value, row r0
        const uint32_t sum_w = smem_u32(row_sum + r0) + quarter * 4;
        // where P's row r0 keeps key j, unswizzled
        const uint32_t p_at = sP + r0 * 128 + (F8 ? j : (j >> 6) * (NP * 128) + (j & 63) * 2);
        bool ok = true;
        int gt = 0, pairs = 0;
        for (; cur.left > 0; ++pairs) {
            const int tiles = cur.run();
            float m[W], l[W], qc[W];
            if constexpr (F8) {
                ok = ok && wait(&bar_q[pairs & 1], (pairs >> 1) & 1, 110, wc);
#pragma unroll
                for (int r = 0; r < W; ++r) qc[r] = q_scale[pairs & 1][r0 + r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_q_free[pairs & 1]);
            }
#pragma unroll
            for (int r = 0; r < W; ++r) {
                m[r] = kNoMax;
                l[r] = 0.0f;
            }
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                const int u = gt + t, s = u % S;
                const int key = (cur.t + t) * kTile + j;
                const int tile_end = (cur.t + t + 1) * kTile;
                const bool tail = tile_end > cur.len;
                // S_u complete means P_{u-2} V_{u-2} complete too: a commit
                // covers every MMA before it, and that one was issued before
                // S_u, so with two buffers P_u's may be written
                ok = ok && (F8 ? wait_both(&bar_s[s], &bar_x[s], (u / S) & 1, 111, wc)
                               : wait(&bar_s[s], (u / S) & 1, 111, wc));
                __syncwarp();
                tc_fence_after();
                uint32_t sa[W], sb[W];
                tmem_ld(lane_base + (u & 1) * N, sa);
                if (F8) tmem_ld(lane_base + (u & 1) * N + RP, sb);
                tmem_ld_done(sa);
                if (F8) tmem_ld_done(sb);
                float ks = 1.0f, vs = 1.0f, lv = 0.0f;
                if constexpr (F8) {
                    ks = lds_f32(sScale + s * C::kScaleBytes + j * 4);
                    vs = lds_f32(sScale + s * C::kScaleBytes + (kTile + j) * 4);
                    if (key >= cur.len) vs = 1.0f;          // may hold anything
                    lv = fmaxf(lg2(fabsf(vs)), kMinLogScale);
                }
                float x[W];
#pragma unroll
                for (int r = 0; r < W; r += 2) {
                    const uint64_t a = pair(sa, r);
                    if constexpr (F8)
                        put(x, r, f2_mul(f2_fma(pair(sb, r), f2(1.0f / C::kQTerm2, 1.0f / C::kQTerm2), a),
                                         f2_mul(pair(qc, r), f2(ks, ks))));
                    else
                        put(x, r, f2_mul(a, f2(p.scale_log2, p.scale_log2)));
                }
                if (tile_end > cur.len - (p.causal ? p.Nq - 1 : 0)) {
#pragma unroll
                    for (int r = 0; r < W; ++r) {
                        const int end = p.causal ? cur.len - p.Nq + 1 + row_query[r0 + r] : cur.len;
                        if (key >= end) x[r] = -CUDART_INF_F;
                    }
                }
                // Does any score pass the reference by 2^kSlack, or may that fall?
                float top = -CUDART_INF_F;
#pragma unroll
                for (int r = 0; r < W; r += 2) {
                    float lo, hi;
                    f2_split(f2_sub(pair(x, r), pair(m, r)), lo, hi);
                    top = W > 1 ? fmax3(top, lo, hi) : lo;
                }
                constexpr int kTurn = C::kRefTiles > 0 ? C::kRefTiles : 1;
                const bool fall = C::kRefTiles > 0 && t > 0 && t % kTurn == 0;
                if (named_bar_or(bar_id, 128, fall || top > C::kSlack - lv)) {
#pragma unroll
                    for (int r = 0; r < W; ++r) {
                        const int y = __reduce_max_sync(0xffffffffu, ordered(x[r] + lv));
                        if (lane == r) sts_u32(max_w + r * 16, __float_as_uint(from_ordered(y)));
                    }
                    named_bar_sync(bar_id, 128);
                    float alpha[W];
#pragma unroll
                    for (int r = 0; r < W; ++r) {
                        const float4 w4 = row_max[r0 + r];
                        float least = m[r];
                        if (fall) {
                            const int turn = t / kTurn;
                            if (turn > 1) least = fmaxf(least, row_top[turn & 1][r0 + r]);
                            if (j == r) row_top[(turn + 1) & 1][r0 + r] = least;
                            least -= C::kRefDrop;
                        }
                        const float mx = fmaxf(fmax3(w4.x, w4.y, w4.z), fmaxf(w4.w, least));
                        alpha[r] = ex2(m[r] - mx);
                        m[r] = mx;
                        l[r] *= alpha[r];
                    }
                    if (t > 0) {
                        ok = ok && wait(&bar_pv[(u - 1) % S], ((u - 1) / S) & 1, 113, wc);
                        __syncwarp();
                        tc_fence_after();
                        if (quarter * 32 < D) {
                            uint32_t oa[W], ob[W];
                            tmem_ld(lane_base + kColO, oa);
                            tmem_ld(lane_base + kColO + RP, ob);
                            tmem_ld_done(oa);
                            tmem_ld_done(ob);
#pragma unroll
                            for (int r = 0; r < W; ++r) {
                                oa[r] = __float_as_uint(__uint_as_float(oa[r]) * alpha[r]);
                                ob[r] = __float_as_uint(__uint_as_float(ob[r]) * alpha[r]);
                            }
                            tmem_st(lane_base + kColO, oa);
                            tmem_st(lane_base + kColO + RP, ob);
                            tmem_st_wait();
                        }
                    }
                }
                // P, at row r's swizzle (its 16-byte units exchanged by r & 7)
                const uint32_t pw = p_at + u % C::kPBufs * C::kPBytes;
                if (C::kPBufs == 1 && u > 0)
                    ok = ok && wait(&bar_pv[(u - 1) % S], ((u - 1) / S) & 1, 118, wc);
                const float wv = vs * C::kPScale;
#pragma unroll
                for (int r = 0; r < W; r += 2) {
                    float e0, e1;
                    f2_split(f2_sub(pair(x, r), pair(m, r)), e0, e1);
                    e0 = ex2(e0);
                    e1 = W > 1 ? ex2(e1) : 0.0f;
                    put(l, r, f2_add(pair(l, r), f2(e0, e1)));
                    const uint32_t a0 = (pw ^ ((r & 7) << 4)) + r * 128;
                    const uint32_t a1 = (pw ^ (((r + 1) & 7) << 4)) + (r + 1) * 128;
                    if constexpr (F8) {
                        // by way of fp16, whose 11 bits hold both terms' 8
                        uint32_t h1, h2;
                        f2_split(f2_mul(f2(e0, e1), f2(wv, wv)), e0, e1);
                        split_e4m3x2(pack_f16x2(e0, e1), h1, h2);
                        sts_u8(a0, h1);
                        sts_u8(a0 + RP * 128, h2);
                        if (W > 1) {
                            sts_u8(a1, h1 >> 8);
                            sts_u8(a1 + RP * 128, h2 >> 8);
                        }
                    } else {
                        const uint32_t h1 = pack_bf16x2(e0, e1);
                        f2_split(f2_sub(f2(e0, e1), f2(__uint_as_float(h1 << 16),
                                                       __uint_as_float(h1 & 0xffff0000u))),
                                 e0, e1);
                        const uint32_t h2 = pack_bf16x2(e0, e1);
                        sts_u16(a0, (uint16_t)h1);
                        sts_u16(a0 + RP * 128, (uint16_t)h2);
                        if (W > 1) {
                            sts_u16(a1, (uint16_t)(h1 >> 16));
                            sts_u16(a1 + RP * 128, (uint16_t)(h2 >> 16));
                        }
                    }
                }
                if (tail && group == 0) {
                    // V rows past the sequence may hold NaN, which a weight
                    // of zero does not silence
                    ok = ok && wait(&bar_v[s], (u / S) & 1, 117, wc);
                    const uint32_t vrow = sKV + s * 2 * TB + j * C::kSw;
#pragma unroll
                    for (int h = 0; h < C::kChunks && key >= cur.len; ++h)
#pragma unroll
                        for (int w = 0; w < C::kSw / 16; ++w)
                            sts_v4(vrow + h * (kTile * C::kSw) + w * 16,
                                   make_uint4(0u, 0u, 0u, 0u));
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&bar_p[u & 1]);
            }
            // The pair's part: O / l, and LSE (or O and LSE themselves).
            int row;
            const float mine = warp_row_sums<W>(l, lane, row);
            sts_u32(sum_w + row * 16, __float_as_uint(mine));    // several lanes, one value
            named_bar_sync(bar_id, 128);
            const int pair = cur.b * p.Hkv + cur.g;
            const bool whole = !CLUSTER && tiles == tiles_of(cur.len);
            const long long out_row = (long long)(whole ? pair : c + pair) * p.R + r0;
            float inv[W], my_l = 0.0f, my_m = 0.0f;
#pragma unroll
            for (int r = 0; r < W; ++r) {
                const float4 w4 = row_sum[r0 + r];
                const float lr = (w4.x + w4.y) + (w4.z + w4.w);
                if (j == r) {
                    my_l = lr;
                    my_m = m[r];
                }
                inv[r] = __fdividef(1.0f, lr * C::kPScale);
                if (lr == 0.0f) inv[r] = -1.0f;                  // saw nothing
            }
            if (j < W && r0 + j < p.R) {
                const float lse2 = my_l == 0.0f ? -CUDART_INF_F : add_log2(my_m, my_l);
                if (CLUSTER)
                    cta_lse[r0 + j] = lse2;
                else if (whole)
                    p.lse[out_row + j] = lse2 * kLn2;
                else
                    p.part_lse[out_row + j] = lse2;
            }
            const int last = gt + tiles - 1;
            ok = ok && wait(&bar_pv[last % S], (last / S) & 1, 115, wc);
            __syncwarp();
            tc_fence_after();
            if (quarter * 32 < D) {
                uint32_t oa[W], ob[W];
                tmem_ld(lane_base + kColO, oa);
                tmem_ld(lane_base + kColO + RP, ob);
                tmem_ld_done(oa);
                tmem_ld_done(ob);
#pragma unroll
                for (int r = 0; r < W; ++r) {
                    float y = fmaf(__uint_as_float(ob[r]), 1.0f / C::kTerm2, __uint_as_float(oa[r]));
                    y = inv[r] < 0.0f ? 0.0f : y * inv[r];
                    if (r0 + r < p.R) {
                        if (CLUSTER)              // P's buffers have been read
                            sts_u32(sP + ((r0 + r) * D + j) * 4, __float_as_uint(y));
                        else if (whole)
                            p.o[(out_row + r) * D + j] = __float2bfloat16_rn(y);
                        else
                            p.part_o[(out_row + r) * D + j] = y;
                    }
                }
            }
            gt += tiles;
            cur.skip(p, tiles);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
    if constexpr (CLUSTER) {
        static_assert(RP * D * 4 <= C::kPBufs * C::kPBytes, "a CTA's part of O in P's buffers");
        // The CTAs deal the rows out among them, D threads a row, one column a
        // thread: every part's LSE and O in one round trip.
        cluster_sync();
        const int j = threadIdx.x % D;
#pragma unroll 1
        for (int r = threadIdx.x / D * p.ctas + cluster_rank(); r < p.R;
             r += C::kThreads / D * p.ctas) {
            float ls[kMaxCluster], y[kMaxCluster], mx = -CUDART_INF_F;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                ls[s] = -CUDART_INF_F;
                y[s] = 0.0f;
                if (s < p.ctas) {
                    ls[s] = ld_cluster_f32(smem_u32(cta_lse + r), s);
                    y[s] = ld_cluster_f32(sP + (r * D + j) * 4, s);
                }
            }
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) mx = fmaxf(mx, ls[s]);
            if (mx == -CUDART_INF_F) mx = 0.0f;
            float sum = 0.0f, acc = 0.0f;
#pragma unroll
            for (int s = 0; s < kMaxCluster; ++s) {
                const float w = ex2(ls[s] - mx);
                sum += w;
                acc = fmaf(w, y[s], acc);         // (s >= p.ctas, or no tiles: w and y are 0)
            }
            const long long row = (long long)c * p.R + r;
            p.o[row * D + j] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : __fdividef(acc, sum));
            if (j == 0) p.lse[row] = sum == 0.0f ? -CUDART_INF_F : add_log2(mx, sum) * kLn2;
        }
        cluster_sync();                           // nobody leaves while its part is read
    }
}

// One warp per query row and 32 columns, for the pairs that several CTAs share:
// the parts weighted by exp(LSE_s - LSE), in slot order.  Rows of empty sequences
// are written here.  Where a row's parts lie follows from the lengths alone and is
// found while the split kernel still runs; after it, the LSEs and the columns of
// 32 parts come in one round trip.
template <int D>
__global__ void __launch_bounds__(256)
fa_paged_combine_kernel(const __grid_constant__ PagedParams p, int rows) {
    constexpr int E = D / 32;                     // warps a row
    pdl_launch_dependents();
    const int at_warp = (int)((blockIdx.x * 256 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    const int row = min(at_warp / E, rows - 1), col = at_warp % E * 32 + lane;
    const int pair = row / p.R, r = row - pair * p.R;
    const int b = pair / p.Hkv, g = pair - b * p.Hkv;
    const List list(p, lane);
    const int tiles = tiles_of(clamped_len(p, b));
    int at = list.at;
#pragma unroll 1
    for (int x = list.b0; x < list.b1 && x < b; ++x) at += list.units_of(p, clamped_len(p, x));
    // from the lane whose sequences b is one of; past the pair's extra unit
    const int first = __shfl_sync(0xffffffffu, at, b / ((p.B + 31) / 32)) +
                      g * (tiles + list.extra) + list.extra;
    const int c0 = tiles ? list.cta_of(first) : 0;
    const int parts = tiles ? list.cta_of(first + tiles - 1) - c0 + 1 : 0;
    // Every thread waits here, also those with nothing to join: this grid must
    // not end before the split kernel, whose results the next one in the
    // stream may read.
    pdl_wait();
    if (at_warp / E >= rows || parts == 1) return;
    const long long slot = (long long)c0 + pair;
    const float* lp = p.part_lse + slot * p.R + r;
    const float* op = p.part_o + (slot * p.R + r) * D + col;
    const long long lstep = p.R, ostep = (long long)p.R * D;
    float mx = -CUDART_INF_F, acc = 0.0f, sum = 0.0f;
#pragma unroll 1
    for (int base = 0; base < parts; base += 32) {
        // this round's parts: LSE of one a lane, its column of each
        const float ls = base + lane < parts ? __ldcg(lp + (base + lane) * lstep) : -CUDART_INF_F;
        float y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; k += 8)
            if (base + k < parts)
#pragma unroll
                for (int i = k; i < k + 8; ++i)
                    if (base + i < parts) y[i] = __ldcg(op + (base + i) * ostep);
        const float top = from_ordered(__reduce_max_sync(0xffffffffu, ordered(ls)));
        const float m = fmaxf(mx, top);
        const float ref = m == -CUDART_INF_F ? 0.0f : m;
        const float old = ex2(mx - ref), w = ex2(ls - ref);
        acc *= old;
        sum = sum * old + w;                      // this lane's parts
#pragma unroll
        for (int k = 0; k < 32; ++k) acc = fmaf(__shfl_sync(0xffffffffu, w, k), y[k], acc);
        mx = m;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    p.o[(long long)row * D + col] =
        __float2bfloat16_rn(sum == 0.0f ? 0.0f : __fdividef(acc, sum));
    if (col == 0)
        p.lse[row] = sum == 0.0f ? -CUDART_INF_F : add_log2(mx, sum) * kLn2;
}

// A launch (in clusters of `cluster` blocks) whose blocks may come in while the
// kernel before in the stream still runs; they wait for it (pdl_wait) before they
// read what it wrote.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kern)(Params...), unsigned grid, unsigned threads, size_t smem,
                       int cluster, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Once a device and kernel: the shared memory it may use.
template <int D, bool F8, int G, int W, bool CLUSTER>
cudaError_t configure(int dev) {
    static std::atomic<unsigned long long> configured{0};     // a bit a device
    if ((configured.load(std::memory_order_acquire) >> dev) & 1) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(fa_decode_paged_kernel<D, F8, G, W, CLUSTER>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg<D, F8, G, W>::kSmem);
    if (e == cudaSuccess) configured.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

// Clusters of 2^log CTAs that the device runs at once (found once a device and
// kernel; 0 where it cannot say).  The SMs of a GPU come in groups that a cluster
// does not cross, so this is less than SMs / size.
template <int D, bool F8, int G, int W>
int clusters_at_once(int dev, int log) {
    using C = Cfg<D, F8, G, W>;
    static std::atomic<int> known[64][4];                     // 1 + the number
    std::atomic<int>& n = known[dev][log];
    if (int k = n.load(std::memory_order_relaxed)) return k - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1u << log);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << log;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int k = 0;
    if (cudaOccupancyMaxActiveClusters(&k, fa_decode_paged_kernel<D, F8, G, W, true>, &cfg) !=
        cudaSuccess)
        k = 0;
    n.store(k + 1, std::memory_order_relaxed);
    return k;
}

template <int D>
cudaError_t launch_combine(const PagedParams& p, cudaStream_t stream) {
    const int rows = p.B * p.Hkv * p.R;
    const long long warps = (long long)rows * (D / 32);
    return launch_pdl(fa_paged_combine_kernel<D>, (unsigned)((warps + 7) / 8), 256, 0, 1, stream,
                      p, rows);
}

template <int D, bool F8, int G, int W>
cudaError_t launch_attend(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                          cudaStream_t stream) {
    using C = Cfg<D, F8, G, W>;
    static_assert(C::kSmem + C::kStatic <= 227 * 1024, "shared memory of one CTA");
    const int longest = ((p.max_pages << p.ps_shift) + kTile - 1) / kTile;    // tiles of a pair
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // Clusters, one a pair, where all of them run at once and leave few tiles to a
    // CTA: the largest size that fits, up to a CTA a tile, or one for every four
    // rows to join (32 rows of 250 keys: 8.1 us with 8 CTAs, 9.0 with a CTA a tile).
    // Smaller ones than eight beat the list too: 16 sequences of 8 kv heads and 250
    // keys 5.5 and 6.3 us, 8 of 1000 keys in e4m3 7.0 and 7.9.
    if (longest <= kMaxCluster * C::kClusterTiles) {
        if ((e = configure<D, F8, G, W, true>(dev)) != cudaSuccess) return e;
        int log = 0;
        while ((1 << log) < max(longest, p.R / 4) && (1 << log) < kMaxCluster) ++log;
        for (; log >= 0 && longest <= C::kClusterTiles << log; --log) {
            if ((long long)p.B * p.Hkv > clusters_at_once<D, F8, G, W>(dev, log)) continue;
            p.ctas = 1 << log;
            return launch_pdl(fa_decode_paged_kernel<D, F8, G, W, true>,
                              (unsigned)(p.B * p.Hkv) << log, C::kThreads, C::kSmem, p.ctas,
                              stream, tk, tv, p);
        }
    }
    if ((e = configure<D, F8, G, W, false>(dev)) != cudaSuccess) return e;
    // no more CTAs than there can be tiles
    const long long most = (long long)p.B * p.Hkv * longest;
    long long grid = (long long)(device_sm_count() > 0 ? device_sm_count() : 152) * C::kCtas;
    if (grid > kPagedMaxCtas) grid = kPagedMaxCtas;
    if (grid > most) grid = most;
    p.ctas = (int)grid;
    e = launch_pdl(fa_decode_paged_kernel<D, F8, G, W, false>, (unsigned)grid, C::kThreads,
                   C::kSmem, 1, stream, tk, tv, p);
    return e == cudaSuccess ? launch_combine<D>(p, stream) : e;
}

template <int D, bool F8>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                        cudaStream_t stream) {
    if (p.R == 1) return launch_attend<D, F8, 1, 1>(tk, tv, p, stream);
    if (p.R <= 4) return launch_attend<D, F8, 1, 4>(tk, tv, p, stream);
    if (p.R <= 8) return launch_attend<D, F8, 1, 8>(tk, tv, p, stream);
    // Two groups of 8 rows rather than one of 16 (e4m3 at d = 128, B8, four tokens, 8K
    // to 16K keys: 41.0 and 42.5 us), two of 16 rather than four of 8 (54.7 and 56.5).
    if (p.R <= 16) return launch_attend<D, F8, 2, 8>(tk, tv, p, stream);
    return launch_attend<D, F8, 2, 16>(tk, tv, p, stream);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t paged_workspace_bytes(int B, int Hkv, int R, int d) {
    const size_t slots = (size_t)kPagedMaxCtas + (size_t)B * Hkv;
    return align256(slots * R * d * 4) + slots * R * 4;
}

cudaError_t launch_fwd_decode_paged(const PagedCache& c, const void* q, void* o, float* lse,
                                    const int* seqlens, void* workspace, int B, int H, int Nq,
                                    int causal, float scale, DeviceStatus* status,
                                    cudaStream_t stream) {
    const bool f8 = c.scales != nullptr;
    const int ps = 1 << c.ps_shift, box = ps < kTile ? ps : kTile;
    CUtensorMap tk, tv;
    if (!make_tmap_pages(&tk, c.k_pages, f8, c.d, ps, (long long)c.n_pages * c.Hkv, box) ||
        !make_tmap_pages(&tv, c.v_pages, f8, c.d, ps, (long long)c.n_pages * c.Hkv, box))
        return cudaErrorInvalidValue;
    PagedParams p;
    p.R = H / c.Hkv * Nq;
    const size_t slots = (size_t)kPagedMaxCtas + (size_t)B * c.Hkv;
    char* ws = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(ws);
    ws += align256(slots * p.R * c.d * 4);
    p.part_lse = reinterpret_cast<float*>(ws);
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.scales = c.scales;
    p.table = c.table;
    p.seqlens = seqlens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.B = B;
    p.Hkv = c.Hkv;
    p.Nq = Nq;
    p.n_pages = c.n_pages;
    p.ps_shift = c.ps_shift;
    p.max_pages = c.max_pages;
    p.causal = causal;
    p.scale_log2 = scale * kLog2e;
    p.status = status;
    if (c.d == 128)
        return f8 ? launch_rows<128, true>(tk, tv, p, stream)
                  : launch_rows<128, false>(tk, tv, p, stream);
    return f8 ? launch_rows<64, true>(tk, tv, p, stream)
              : launch_rows<64, false>(tk, tv, p, stream);
}

}  // namespace fa
