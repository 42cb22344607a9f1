// Forward kernel: exact attention with the online-softmax recurrence, tiled so
// the N x N score matrix never leaves the SM (FlashAttention blog, "From Online
// Softmax to FlashAttention" and "FlashAttention"; FlashAttention-2 review
// thread, author answers on non-matmul FLOPs and on Figure 2).
//
// Persistent grid, one CTA per SM.  A work item is two 128-row query tiles
// (t = 0, 1) of one (batch, head); CTA c takes items c, c + gridDim.x, ...
// (longest causal items first) and streams 128-key K and V tiles through two
// shared-memory rings:
//   warp 8      TMA producer of K_j; K_j is released when both S MMAs that
//               read it have completed, so K loads run whole blocks ahead.
//               In the PRECISE variant the whole warp also re-encodes the
//               second half of each landed V_j as fp16, in place.
//   warp 10     TMA producer of V_j and of the Q tiles (each item's Q ahead of
//               its V blocks); V_j is released after both P V MMAs.  In the
//               PRECISE variant the whole warp also re-encodes the first half
//               of each landed V_j as fp16, in place.
//   warp 9      S MMA issuer (one thread): S_t = Q_t K_j^T into TMEM (SS MMA).
//   warp 11     P V MMA issuer (one thread): O_t += P_t V_j, P_t read from
//               TMEM (TS MMA).  An MMA issue blocks while the tensor pipe is
//               busy, and every barrier wait, fence and commit of an issuing
//               thread costs on the order of a hundred cycles; with two
//               issuers one thread's waits overlap the other's MMAs.
//   warps 0-3   softmax for tile 0, warps 4-7 for tile 1: one query row per
//               thread.  While one group does its softmax the tensor core
//               runs the other tile's MMAs.
// TMEM (512 columns): S_0 | S_1 | O_0 | O_1.  At d = 128, P_t (bf16 pairs)
// overwrites the first half of S_t; the MMA that next writes S_t is issued
// only after the P_t V MMA that reads P_t has completed.
// At d = 64 (bf16 output) P_t has columns of its own after O_1, which breaks
// that chain: the softmax releases S_t as soon as it has loaded it, the next
// S_t MMA is issued at once, and the softmax waits for the previous P V MMA
// only just before it writes P_t.  The tensor core then works on S_t(j+1) and
// P_t(j-1) V while the softmax of block j runs.
//
// Softmax in base 2: p = 2^(S*c - m) with c = scale*log2(e).  The running max
// m is only raised when the block max exceeds it by more than 8 (a factor
// 256), so most blocks skip the O rescale; numerator and denominator always
// use the same m, so the result is unchanged in exact arithmetic.  O is
// divided by l once, in the epilogue, and LSE = ln2 * (m + log2 l).
//
// PRECISE variant: the P V product runs in fp16 instead of bf16 (same tensor
// rate): P is rounded to fp16 (11 significant bits against bf16's 8), V_j is
// re-encoded as fp16 in shared memory (exact for magnitudes in [2^-14,
// 65280]; 65536 and above overflow to infinity), and O is written in fp32.
// This takes the bf16 rounding of O out of the error (half a bf16 ulp of 30 is
// 0.06) and cuts that of P eightfold: each p is off by at most 2^-11 of
// itself (2^-25 absolute below 2^-14).  The row sum l is corrected by what
// the rounding added to each key block's largest p, so a row whose weight
// sits on one key returns that key's V row unrounded; in general a row of O
// moves by at most 2^-11 (sum over block maxima of w |v - O| + sum over the
// other keys of w |v|) <= 2^-10 max|V|, w = p / l.
#include <cuda_bf16.h>
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kBM = 128;          // query rows per tile
constexpr int kBN = 128;          // keys per K/V tile
constexpr int kTiles = 2;         // query tiles per CTA
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 12 * 32;   // 3 warpgroups: softmax 0, softmax 1, control
constexpr int kProducerWarp = 8;    // K tiles
constexpr int kMmaWarp = 9;
constexpr int kVProducerWarp = 10;  // V and Q tiles
constexpr int kPvWarp = 11;         // P V MMA issuer
// Register split (setmaxnreg): the launch gives 384 x 168; the control
// warpgroup drops to 72 so each softmax thread can hold a full 128-score row:
// 128 x 72 + 256 x 216 = 64512 <= 384 x 168 = 64512.  At 216 no role spills
// (at 208 the softmax warps did, d = 128: forward 3 % slower).
constexpr int kRegsControl = 72;
constexpr int kRegsSoftmax = 216;
constexpr int kRegsNeeded = 128 * kRegsControl + 256 * kRegsSoftmax;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
// One pair in every kExp2FmaEvery of a row's exps is computed on the FMA pipe
// (exp2_fma2) instead of the exponential unit, 0 = none.  Measured on the
// forward alone: d = 128 one pair in 8: +1.8 % (one in 16 +0.6 %, one in 4
// -4.6 %); d = 64, where the softmax is bound by instruction issue rather than
// by the exponential unit: one in 16 -4 %, one in 8 -6.5 %.
template <int D, bool PRECISE>
struct Exp2FmaEvery {
    static constexpr int value = (D == 128 && !PRECISE) ? 8 : 0;
    static constexpr int mod = value > 0 ? value : 1;
};

template <int D, bool PRECISE = false>
struct FwdCfg {
    // K and V have rings of their own: K is released as soon as both S MMAs of
    // a block are issued, V after both P V MMAs.  The PRECISE variant holds
    // each V_j longer (its fp16 re-encoding sits between landing and use) and
    // at d = 128 trades a K stage for a third V stage.
    static constexpr int kStagesK = (D == 128) ? (PRECISE ? 2 : 3) : 4;
    static constexpr int kStagesV = (D == 128) ? (PRECISE ? 3 : 2) : 3;
    static constexpr int kTileBytes = kBM * D * 2;          // one Q, K or V tile
    static constexpr int kChunks = D / 64;                  // 128-byte swizzle chunks
    static constexpr int kChunkBytes = 128 * 128;           // 128 rows x 128 bytes
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kTiles * kTileBytes;
    static constexpr int kOffV = kOffK + kStagesK * kTileBytes;
    static constexpr int kSmemBytes = kOffV + kStagesV * kTileBytes;
    static constexpr int kSmemAlloc = kSmemBytes + 1024;    // alignment slack
    // TMEM columns
    static constexpr uint32_t kColS0 = 0, kColS1 = 128, kColO0 = 256, kColO1 = 256 + D;
    // At d = 64, S_0 | S_1 | O_0 | O_1 fill 384 columns and P_t (64 columns of
    // bf16 pairs) gets columns of its own.
    static constexpr uint32_t kColP0 = 384, kColP1 = 448;
};

// A place in the list of (item, key block) of a forward with keys of its own: block blk
// of item it of sequence b.
struct CrossAt {
    int b, it, blk, pad;
};

struct FwdParams {
    int H, Hkv, N, BH, n_mblk, n_items, causal;
    // Causal sliding window W: query i sees keys i - W < j <= i.  Without a
    // window this holds kNoWindow, so large that the lower edge never binds.
    int window;
    // Packed variable-length batches: sequence b is rows cu_seqlens[b] ..
    // cu_seqlens[b+1] - 1 of every head ([H][rows][d]); N is then the
    // longest sequence.  Dense batches: rows = N, cu_seqlens unused.
    int rows;
    const int* cu_seqlens;
    // Keys of their own (CROSS): at most Nk of them a sequence, krows rows a head of
    // k and v.  Padded batches: kv_lens[b] of them, or Nk (null).  Packed ones: rows
    // cu_k[b] .. cu_k[b+1] - 1.
    int Nk, krows;
    const int* kv_lens;
    const int* cu_k;
    // CROSS: may key blocks of one item go to several CTAs?  Then the segments' places
    // in the workspace: [slot][d / 4][256 rows] quarter rows of O (normalised, fp32),
    // [slot][256] LSEs (base 2), and where each CTA's part begins.
    int split;
    float4* part_o;
    float* part_lse;
    CrossAt* part_at;
    float scale_log2;                 // scale * log2(e)
    void* o;                          // bf16, or fp32 in the precise variant
    float* lse;
    DeviceStatus* status;
    // Training forward (dense batches): the backward workspace rows this
    // forward prepares, Np (= N rounded up to 128) rows per (batch, head):
    // the -LSE table row and a zeroed dQ accumulator row.  nullptr = none.
    uint16_t* lse_ext;
    float* dq_acc;
    int Np;
};

// Work item (query-block pair, batch*head) -> coordinates.  Under the causal
// mask the longest query blocks come first (the tile list is in decreasing
// cost order, and each CTA takes every gridDim.x-th item).
struct FwdTile {
    int bh, row_base;
    int q_z, kv_z;             // head coordinate of the Q / O and K / V tensor maps
    int tok0, len;             // first row of the sequence in its head, its length
    int ktok0, klen;           // the same of its keys
    int off;                   // query i sees keys j <= i + off under the causal mask
    int lo[kTiles];            // first key block each query tile needs
    int n_kv[kTiles];          // one past its last key block
};
struct CrossTile : FwdTile {
    int slot;                  // of a segment of an item, else -1
};

// The keys of sequence b (CROSS): how many, and the first one's row in its head.
__device__ __forceinline__ int key_rows(const FwdParams& p, int b, int& ktok0) {
    if (p.cu_k) return packed_seq(p.cu_k, b, p.Nk, p.krows, ktok0);
    ktok0 = 0;
    return p.kv_lens ? min(max(__ldg(p.kv_lens + b), 0), p.Nk) : p.Nk;
}

__device__ __forceinline__ int fwd_m_blk(int item, const FwdParams& p, bool causal) {
    const int mb_rank = item / p.BH;
    return causal ? (p.n_mblk - 1 - mb_rank) : mb_rank;
}

// The work items of this CTA, the same sequence for every role.  Items are
// ranked in decreasing cost (under the causal mask) and dealt out in rounds
// of gridDim.x, the order of the CTAs reversed every other round ("snake"),
// so that the sum of costs per CTA evens out (CPU model of the bench
// workloads: 0.98-1.00 of the mean load per CTA, against 0.88-0.94 for
// plain round robin).  With variable lengths the ranks count only the items
// that have rows (query-block pairs past a sequence's end are passed over):
// a cursor walks the (level, sequence) list forward, ranks only grow.
template <bool VARLEN, bool CROSS>
struct FwdSched {
    int round = 0;
    int mb = 0, b = 0, base = 0;   // cursor: level, sequence, rank of (b, head 0)

    __device__ __forceinline__ int next(const FwdParams& p, bool causal) {
        const int G = gridDim.x, c = blockIdx.x;
        const int t = round * G + ((round & 1) ? G - 1 - c : c);   // rank
        ++round;
        if (!VARLEN) return t < p.n_items ? t : p.n_items;
        const int B = p.BH / p.H;
        while (mb < p.n_mblk) {
            if (b >= B) {
                ++mb;
                b = 0;
                continue;
            }
            int t0;
            const int len = packed_seq(p.cu_seqlens, b, p.N, p.rows, t0);
            if (fwd_m_blk(mb * p.BH, p, causal) * (kTiles * kBM) < len) {
                if (t < base + p.H) return mb * p.BH + b * p.H + (t - base);
                base += p.H;
            }
            ++b;
        }
        return p.n_items;
    }
};

// Keys of another length (CROSS).  The work is a list of (item, key block): sequences in
// turn, in each the K/V heads, in each the query-block pairs, in each the query heads that
// share the K/V head, and the item's key blocks.  Each CTA takes an equal share of that
// list, whole items or segments of them; an item in segments leaves one partial result
// each in the workspace (a CTA has two at most: its first and its last item), which
// cross_join_kernel adds up in the order of the keys.  The lengths are on the device, so
// that each CTA finds its share itself.  Whole items in rounds leave the GPU idle in the
// last one and are as long as the longest sequence allows: 2 x 32/8 heads, 1024 queries,
// 17408 keys, d = 128, causal (256 items on 152 SMs): 437 us, in equal shares 390 to 410.
// Segments pay for the join (a launch, 132 KB written and read each at d = 128): about
// kJoinCost key blocks, so that cross_ctas() takes them only where an even share is that
// much shorter; a segment has kMinBlocks blocks at least, and a share that would end
// within 1/24 of itself of an item's end ends there.  8 heads, 64 queries, d = 128, whole
// items against segments: 1024 keys 20.6 us / 17.8, 16384 keys 200 / 35; 4 x 32 heads, 256
// queries (128 items): 2048 keys 40.0 / 48.8, which the rule leaves whole.
constexpr int kSplitBlocks = 4;   // no segments up to here
constexpr int kMinBlocks = 2;
constexpr int kJoinCost = 8;
constexpr int kItemCost = 3;      // what an item costs besides its key blocks, in those
constexpr int kMaxCtas = 152;     // the workspace has places for that many

// The items of sequence b, and the key blocks of each.
struct CrossSeq {
    int tok0, len, ktok0, klen;
    int M, n;         // query-block pairs; key blocks
    int q;            // causal: pair m sees 2 (m + 1) + q of them
    bool causal;

    __device__ __forceinline__ CrossSeq(const FwdParams& p, int b, bool causal_) {
        if (p.cu_seqlens) {
            len = packed_seq(p.cu_seqlens, b, p.N, p.rows, tok0);
        } else {
            tok0 = 0;
            len = p.N;
        }
        klen = key_rows(p, b, ktok0);
        causal = causal_;
        M = (len + kTiles * kBM - 1) / (kTiles * kBM);
        n = max(1, (klen + kBN - 1) / kBN);
        q = (klen - len + kBN - 1) >> 7;   // rounds down for negative ones too
    }
    __device__ __forceinline__ int blocks(int m) const {
        return causal ? min(max(2 * (m + 1) + q, 1), n) : n;
    }
    // Cost of pairs 0 .. m - 1, key blocks and kItemCost each: pairs below m1 have one
    // block, those from m2 on all n.
    __device__ __forceinline__ long long before(int m) const {
        if (!causal) return (long long)m * (n + kItemCost);
        const int m1 = min(max((1 - q) >> 1, 0), m);
        const int m2 = min(max((n - q) >> 1, m1), m);
        const long long mid = m2 - m1;
        return m1 + mid * (m1 + m2 + 1 + q) + (long long)(m - m2) * n + (long long)m * kItemCost;
    }
};
static_assert(kBN == 128 && kBM == 128 && kTiles == 2, "CrossSeq counts in these");

// First block of CTA c's share: block t of the list, which lies in sequence b at o.
__device__ __forceinline__ CrossAt cross_place(const FwdParams& p, const CrossSeq& sq, int b,
                                               long long o, bool unit, int snap) {
    const int G = p.H / p.Hkv;
    CrossAt at;
    at.b = b;
    if (unit) {   // every item counts as one
        at.it = (int)o;
        at.blk = 0;
        return at;
    }
    const long long head = G * sq.before(sq.M);
    const int g = o >> 31 ? (int)(o / head) : (int)((uint32_t)o / (uint32_t)min(head, 0x7fffffffll));
    o -= g * head;
    int m = 0;                          // the last pair with G before(m) <= o
    for (int hi = sq.M; hi - m > 1;) {
        const int mid = (m + hi) >> 1;
        if (G * sq.before(mid) <= o) m = mid;
        else hi = mid;
    }
    o -= G * sq.before(m);
    const int n = sq.blocks(m), cost = n + kItemCost, r = (int)o / cost;
    at.it = (g * sq.M + m) * G + r;
    at.blk = max((int)o - r * cost - kItemCost, 0);
    if (at.blk <= snap && (p.split || 2 * at.blk < n)) {
        at.blk = 0;
    } else if (n - at.blk <= snap) {
        at.blk = 0;
        if (++at.it == p.H * sq.M) {
            ++at.b;
            at.it = 0;
        }
    }
    return at;
}

// The block's share [at[0], at[1]): every thread counts the blocks of a run of sequences.
__device__ __forceinline__ void cross_share(const FwdParams& p, bool causal, CrossAt* at,
                                            long long* warp_sum) {
    const int B = p.BH / p.H;
    const int run = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, (int)threadIdx.x * run), b1 = min(B, b0 + run);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool unit = !p.split && p.n_items <= (int)gridDim.x;
    auto count = [&](const CrossSeq& sq) -> long long {
        return p.H * (unit ? (long long)sq.M : sq.before(sq.M));
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += count(CrossSeq(p, b, causal));
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) upto += total;
        total += warp_sum[w];
    }
    const long long per = max((total + gridDim.x - 1) / gridDim.x,
                              (long long)(p.split ? kMinBlocks : 1));
    // whole items: the nearest item's end
    const int snap = p.split ? (int)max(1ll, min(per / 24, 1ll << 20)) : 1 << 30;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const long long t = ((long long)blockIdx.x + e) * per;
        if (t >= total) {
            if (threadIdx.x == 0) at[e] = CrossAt{B, 0, 0, 0};
        } else if (t >= upto - mine && t < upto) {
            long long o = t - (upto - mine);
            for (int b = b0; b < b1; ++b) {
                const CrossSeq sq(p, b, causal);
                const long long n = count(sq);
                if (o < n) {
                    at[e] = cross_place(p, sq, b, o, unit, snap);
                    break;
                }
                o -= n;
            }
        }
    }
}

// The CTA's items and segments.  The K producer, which is ahead of every other role, finds
// them and leaves them in a ring in shared memory (struct CrossRing): found by each role
// by itself, with divisions and loads in one thread, an item cost 2 to 4 us more than one
// of a dense batch (d = 64 to 128).
struct CrossWalk {
    const CrossAt* at;   // shared memory: the share's first place and its end
    int b, it, blk;      // the item, and the first block of it
    bool begun = false;

    __device__ __forceinline__ explicit CrossWalk(const CrossAt* a)
        : at(a), b(a[0].b), it(a[0].it), blk(a[0].blk) {}

    __device__ __forceinline__ bool next(const FwdParams& p, bool causal) {
        if (begun) {
            ++it;
            blk = 0;
        }
        begun = true;
        for (;;) {
            if (b > at[1].b || (b == at[1].b && it > at[1].it)) return false;
            if (b == at[1].b && it == at[1].it) return at[1].blk > blk;
            if (it < p.H * CrossSeq(p, b, causal).M) return true;
            ++b;
            it = 0;
        }
    }
};

__device__ __forceinline__ CrossTile cross_tile(const CrossWalk& sch, const FwdParams& p,
                                                bool causal) {
    const CrossSeq sq(p, sch.b, causal);
    const int G = p.H / p.Hkv;
    const int m = sch.it / G % sq.M, kv = sch.it / G / sq.M, h = kv * G + sch.it % G;
    CrossTile w;
    w.bh = sch.b * p.H + h;
    w.tok0 = sq.tok0;
    w.len = sq.len;
    w.ktok0 = sq.ktok0;
    w.klen = sq.klen;
    w.off = sq.klen - sq.len;
    w.q_z = p.cu_seqlens ? h : w.bh;
    w.kv_z = p.cu_seqlens ? kv : sch.b * p.Hkv + kv;
    w.row_base = m * (kTiles * kBM);
    const int n = sq.blocks(m);
    const int lo = sch.blk;
    const int hi = sch.b == sch.at[1].b && sch.it == sch.at[1].it ? sch.at[1].blk : n;
    // The first tile's last row sees keys up to its own index + off.  A tile that sees
    // nothing of the segment keeps one block, which the masks empty.
    const int n0 = causal ? min(n, max(2 * m + 1 + sq.q, 1)) : n;
    w.lo[0] = w.lo[1] = lo;
    w.n_kv[0] = max(lo + 1, min(n0, hi));
    w.n_kv[1] = hi;
    // (its first item may lack a beginning, its last one an end)
    w.slot = lo > 0 ? 2 * (int)blockIdx.x : hi < n ? 2 * (int)blockIdx.x + 1 : -1;
    return w;
}

constexpr int kRing = 4;
constexpr int kRingReaders = 3 + 8;   // V producer, the two issuers, the softmax warps

struct CrossRing {
    CrossTile tile[kRing];   // n_kv[1] == 0: no more
    uint64_t full[kRing], empty[kRing];
};

// A reader's way through the ring, by one thread or (warp) a whole warp.
template <bool VARLEN>
struct FwdSched<VARLEN, true> {
    CrossRing* ring;
    WaitCtx wc;
    bool warp;
    uint32_t i = 0;
    bool ok = true;

    __device__ __forceinline__ const CrossTile& tile() const { return ring->tile[(i - 1) % kRing]; }
    // An index below p.n_items (0) while there is one more: tile() is it until the next call.
    __device__ __forceinline__ int next(const FwdParams& p, bool) {
        if (i > 0) {
            if (warp) __syncwarp();
            if (!warp || (threadIdx.x & 31) == 0) mbar_arrive(&ring->empty[(i - 1) % kRing]);
        }
        uint64_t* full = &ring->full[i % kRing];
        const uint32_t par = (i / kRing) & 1;
        ok = warp ? fa_wait_warp(full, par, 40, wc) : fa_wait(full, par, 40, wc);
        ++i;
        return ok && tile().n_kv[kTiles - 1] > 0 ? 0 : p.n_items;
    }
};

template <bool WINDOW, bool VARLEN>
__device__ __forceinline__ FwdTile fwd_tile(int item, const FwdParams& p, bool causal) {
    FwdTile w;
    w.bh = item % p.BH;
    const int m_blk = fwd_m_blk(item, p, causal);
    const int b = w.bh / p.H, h = w.bh % p.H;
    if (VARLEN) {
        w.len = packed_seq(p.cu_seqlens, b, p.N, p.rows, w.tok0);
        w.q_z = h;
        w.kv_z = h / (p.H / p.Hkv);
    } else {
        w.tok0 = 0;
        w.len = p.N;
        w.q_z = w.bh;
        w.kv_z = b * p.Hkv + h / (p.H / p.Hkv);
    }
    w.ktok0 = w.tok0;
    w.klen = w.len;
    w.off = 0;
    w.row_base = m_blk * (kTiles * kBM);
    const int n_kv_all = (w.klen + kBN - 1) / kBN;
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        w.n_kv[t] = causal ? min(n_kv_all, 2 * m_blk + t + 1) : n_kv_all;
        // The tile's first row sees keys from row0 - W + 1 on.  A tile wholly
        // past N (the second tile of the last pair) keeps one block, which
        // the masks empty, so that every tile takes at least one block.
        w.lo[t] = WINDOW ? min(max(0, w.row_base + t * kBM - p.window + 1) / kBN, w.n_kv[t] - 1)
                         : 0;
    }
    return w;
}

// WINDOW (with CAUSAL): the causal sliding window of p.window keys.
// VARLEN: packed variable-length sequences (p.cu_seqlens).
// PRECISE: one warp's half (part 0 or 1) of the fp16 re-encoding of V_x, in
// place, once V_x has landed; the P V issuer waits for both halves (bar_v_cvt
// counts two arrivals).  Spread over two warps on two SM sub-partitions, the
// conversion takes issue slots from fewer softmax warps each.
template <int SV, int TILE_BYTES>
__device__ __forceinline__ bool convert_v_half(uint8_t* sV, uint64_t* bar_v, uint64_t* bar_v_cvt,
                                               uint32_t x, int part, int lane, const WaitCtx& wc) {
    const uint32_t s = x % SV;
    if (!fa_wait_warp(&bar_v[s], (x / SV) & 1, 16 + part, wc)) return false;
    constexpr int kHalf = TILE_BYTES / 32;   // 16-byte pieces in half a tile
    uint4* v4 = reinterpret_cast<uint4*>(sV + s * TILE_BYTES) + part * kHalf;
#pragma unroll 8
    for (int i = lane; i < kHalf; i += 32) {
        uint4 w = v4[i];
        w.x = bf16x2_to_f16x2(w.x);
        w.y = bf16x2_to_f16x2(w.y);
        w.z = bf16x2_to_f16x2(w.z);
        w.w = bf16x2_to_f16x2(w.w);
        v4[i] = w;
    }
    fence_proxy_async_smem();   // visible to the tensor core's reads
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_v_cvt[s]);
    return true;
}

// CROSS: queries against keys of another length (p.Nk, p.kv_lens, p.cu_k), padded or
// packed (p.cu_seqlens), the causal mask by p.causal and counted from the last key.
// Rows past a sequence's keys may hold anything: their scores are masked, and the
// softmax of query tile 0 (of tile 1 where only that sees the block) clears V's rows.
template <int D, bool CAUSAL, bool PRECISE, bool WINDOW, bool VARLEN, bool CROSS>
__global__ void __launch_bounds__(kThreads, 1)
fa_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
    using Cfg = FwdCfg<D, PRECISE>;
    constexpr int SK = Cfg::kStagesK, SV = Cfg::kStagesV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bar_k[SK], bar_k_empty[SK], bar_v[SV], bar_v_empty[SV];
    __shared__ uint64_t bar_v_cvt[SV];        // PRECISE: V_j re-encoded as fp16
    __shared__ uint64_t bar_q[kTiles], bar_q_free[kTiles];
    __shared__ uint64_t bar_s[kTiles], bar_p[kTiles], bar_pv[kTiles], bar_o_free[kTiles];
    __shared__ uint64_t bar_s_free[kTiles];   // separate-P form only
    constexpr bool SEP = (D == 64) && !PRECISE;
    constexpr int kExp2FmaEvery = Exp2FmaEvery<D, PRECISE>::value;
    constexpr int kExp2FmaMod = Exp2FmaEvery<D, PRECISE>::mod;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    const WaitCtx wc{p.status, &abort_sh};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool causal = CAUSAL || (CROSS && p.causal);
    __shared__ CrossAt share[2];
    __shared__ CrossRing ring;
    auto sched = [&](bool whole_warp) {
        if constexpr (CROSS) return FwdSched<VARLEN, CROSS>{&ring, wc, whole_warp};
        else return FwdSched<VARLEN, CROSS>();
    };
    auto tile = [&](int item, const FwdSched<VARLEN, CROSS>& sch) {
        if constexpr (CROSS) return static_cast<FwdTile>(sch.tile());
        else return fwd_tile<WINDOW, VARLEN>(item, p, causal);
    };
    if constexpr (CROSS) {
        __shared__ long long warp_sum[kThreads / 32];
        cross_share(p, causal, share, warp_sum);
    }

    if (threadIdx.x == 0) {
        abort_sh = 0;
        for (int s = 0; s < SK; ++s) {
            mbar_init(&bar_k[s], 1);
            mbar_init(&bar_k_empty[s], 1);
        }
        for (int s = 0; s < SV; ++s) {
            mbar_init(&bar_v[s], 1);
            mbar_init(&bar_v_empty[s], 1);
            mbar_init(&bar_v_cvt[s], 2);   // one arrival per converting warp
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&bar_q[t], 1);
            mbar_init(&bar_q_free[t], 1);
            mbar_init(&bar_s[t], 1);
            mbar_init(&bar_p[t], 128);
            mbar_init(&bar_o_free[t], 128);
            mbar_init(&bar_s_free[t], 128);
            mbar_init(&bar_pv[t], 1);
        }
        if constexpr (CROSS)
            for (int r = 0; r < kRing; ++r) {
                mbar_init(&ring.full[r], 1);
                mbar_init(&ring.empty[r], kRingReaders);
            }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    uint8_t* sQ = smem + Cfg::kOffQ;
    uint8_t* sK = smem + Cfg::kOffK;
    uint8_t* sV = smem + Cfg::kOffV;

    // One register-budget change per warpgroup, executed by all its warps at
    // the same instruction; each role's code is dominated by exactly one.
    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2;                 // query tile of this group
        const int quarter = warp & 3;            // TMEM lane quarter
        const int rl = quarter * 32 + lane;      // row within the tile
        const uint32_t col_s = t ? Cfg::kColS1 : Cfg::kColS0;
        const uint32_t col_o = t ? Cfg::kColO1 : Cfg::kColO0;
        const uint32_t col_p = SEP ? (t ? Cfg::kColP1 : Cfg::kColP0) : col_s;
        const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
        const float c = p.scale_log2;
        uint32_t cs = 0;                         // S_t completions seen so far
        uint32_t cpv = 0;                        // P_t V completions seen (separate P)
        uint32_t gv = 0;                         // V blocks of the items before (CROSS)
        bool ok = true;
        int lt = 0;
        FwdSched<VARLEN, CROSS> sch = sched(true);
        for (int item = sch.next(p, causal); ok && item < p.n_items;
             item = sch.next(p, causal), ++lt) {
            const FwdTile wt = tile(item, sch);
            const int row0 = wt.row_base + t * kBM;
            const int row = row0 + rl;
            // (selects, not a run-time index: the arrays stay in registers)
            const int lo = t ? wt.lo[1] : wt.lo[0], n_kv = t ? wt.n_kv[1] : wt.n_kv[0];
            float m2 = -CUDART_INF_F;   // running max, log2-scaled
            float l = 0.0f;
            // PRECISE: what the fp16 rounding of each block's largest p added
            // to the P V product, scaled like l.  O is divided by l + lc, so a
            // row whose weight sits on one key returns that key's V row
            // without the rounding of its p (up to 2^-11 |V| otherwise); the
            // LSE keeps l.
            float lc = 0.0f;
            for (int j = lo; j < n_kv; ++j) {
                if (CROSS && (j + 1) * kBN > wt.klen && (t == 0 || j >= wt.n_kv[0])) {
                    // V_j's rows past the keys: a weight of zero would not silence a
                    // NaN.  Before the scores are waited for (the loads of V_j wait for
                    // none of this tile's MMAs to come), and by the stage's order no
                    // other use of the stage comes before this tile's P V.
                    const uint32_t gj = gv + (uint32_t)(j - lo), vs = gj % SV;
                    if (!fa_wait_warp(&bar_v[vs], (gj / SV) & 1, 38 + t, wc)) { ok = false; break; }
                    if (j * kBN + rl >= wt.klen) {
                        const uint32_t vrow = smem_u32(sV) + vs * Cfg::kTileBytes + rl * 128;
#pragma unroll
                        for (int u = 0; u < Cfg::kChunks * 8; ++u)   // (eight lanes, eight banks)
                            sts_v4(vrow + (u >> 3) * Cfg::kChunkBytes + ((u ^ rl) & 7) * 16,
                                   make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_smem();
                }
                if (!fa_wait_warp(&bar_s[t], cs & 1, 30 + t, wc)) { ok = false; break; }
                ++cs;
                tc_fence_after();
                uint32_t r[4][32];
                tmem_ld32(lane_addr + col_s + 0, r[0]);
                tmem_ld32(lane_addr + col_s + 32, r[1]);
                tmem_ld32(lane_addr + col_s + 64, r[2]);
                tmem_ld32(lane_addr + col_s + 96, r[3]);
                tmem_ld_wait(r[0]);
                asm volatile("" : FA_R32(r[1]) : : "memory");
                asm volatile("" : FA_R32(r[2]) : : "memory");
                asm volatile("" : FA_R32(r[3]) : : "memory");
                if (SEP) {   // S_t is in registers: the next S_t MMA may overwrite it
                    tc_fence_before();
                    mbar_arrive(&bar_s_free[t]);
                }
                float sv[kBN];
#pragma unroll
                for (int e = 0; e < kBN; ++e) sv[e] = __uint_as_float(r[e >> 5][e & 31]);

                const int col0 = j * kBN;
                const bool need_mask = (causal && (col0 + kBN - 1 > row0 + wt.off ||
                                                   (WINDOW && col0 < row0 + kBM - p.window))) ||
                                       (col0 + kBN > wt.klen);
                if (need_mask) {
                    const int lim_causal = causal ? row + wt.off - col0 : kBN;   // keep e <= this
                    const int lim_n = wt.klen - col0;                    // keep e < N - col0
                    if (CROSS) {
                        const int lim = min(lim_causal, lim_n - 1);
#pragma unroll
                        for (int e = 0; e < kBN; ++e)
                            if (e > lim) sv[e] = -CUDART_INF_F;
                    } else {
                        const int lim_lo = WINDOW ? row - p.window + 1 - col0 : 0;  // keep e >= this
#pragma unroll
                        for (int e = 0; e < kBN; ++e)
                            if (e > lim_causal || e >= lim_n || e < lim_lo) sv[e] = -CUDART_INF_F;
                    }
                }
                // Row max: three-input max, eight independent chains.
                float mx8[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) mx8[u] = fmaxf(sv[2 * u], sv[2 * u + 1]);
#pragma unroll
                for (int e = 16; e < kBN; e += 16)
#pragma unroll
                    for (int u = 0; u < 8; ++u) mx8[u] = fmax3(mx8[u], sv[e + 2 * u], sv[e + 2 * u + 1]);
                const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]),
                                       fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
                const float mx2 = mx * c;
                const bool need = mx2 > m2 + kRescaleThreshold;
                // O rescale of this block (only when some row raised its max);
                // the O columns may be touched only after the P V MMA of the
                // previous block has completed.
                auto rescale_o = [&](float alpha) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32(lane_addr + col_o + c0, ov);
                        tmem_ld_wait(ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tmem_st32(lane_addr + col_o + c0, ov);
                    }
                };
                const bool any_need = __any_sync(0xffffffffu, need);
                float alpha = 1.0f;
                if (any_need) {
                    const float m_new = need ? mx2 : m2;
                    alpha = (m_new == m2) ? 1.0f : ex2(m2 - m_new);
                    l *= alpha;
                    if (PRECISE) lc *= alpha;
                    if (!SEP && j > lo) rescale_o(alpha);
                    m2 = m_new;
                }
                const float m_use = (m2 == -CUDART_INF_F) ? 0.0f : m2;
                if (PRECISE) {   // the block max's p, as the loop below computes it
                    const float pm = ex2(fmaf(mx, c, -m_use));
                    float h0, h1;
                    unpack_f16x2(pack_f16x2(pm, 0.0f), h0, h1);
                    lc += h0 - pm;
                }
                // p = 2^(s c - m): exponent argument two lanes per instruction,
                // row sum in four paired accumulators.
                const uint64_t c2 = f2(c, c), negm2 = f2(-m_use, -m_use);
                uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t pk[2][32];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                    for (int e2 = 0; e2 < 32; ++e2) {
                        const int e = hh * 64 + 2 * e2;
                        float p0, p1;
                        if (kExp2FmaEvery > 0 && e2 % kExp2FmaMod == kExp2FmaMod - 1) {
                            // this pair on the FMA pipe (exp2_fma2), the rest
                            // on the exponential unit
                            f2_split(exp2_fma2(f2_fma(f2(sv[e], sv[e + 1]), c2, negm2)), p0, p1);
                        } else {
                            float x0, x1;
                            f2_split(f2_fma(f2(sv[e], sv[e + 1]), c2, negm2), x0, x1);
                            p0 = ex2(x0);
                            p1 = ex2(x1);
                        }
                        acc2[e2 & 3] = f2_add(acc2[e2 & 3], f2(p0, p1));
                        pk[hh][e2] = PRECISE ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                    }
                    if (!SEP) tmem_st32(lane_addr + col_s + hh * 32, pk[hh]);
                }
                if (SEP) {
                    // P_t and O_t are free once P_t(j-1) V has completed.
                    if (j > lo) {
                        if (!fa_wait_warp(&bar_pv[t], cpv & 1, 34 + t, wc)) { ok = false; break; }
                        ++cpv;
                        tc_fence_after();
                        if (any_need) rescale_o(alpha);
                    }
                    tmem_st32(lane_addr + col_p, pk[0]);
                    tmem_st32(lane_addr + col_p + 32, pk[1]);
                }
                {
                    float a0, a1;
                    f2_split(f2_add(f2_add(acc2[0], acc2[1]), f2_add(acc2[2], acc2[3])), a0, a1);
                    l += a0 + a1;
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&bar_p[t]);
            }
            if (!ok) break;
            if (CROSS) gv += wt.n_kv[kTiles - 1] - lo;

            // ------------------------------------------------------- epilogue
            // O row -> registers, release the O columns to the next item's
            // MMAs, then normalise and store.
            // The last P_t V MMA of the item has completed.  Without separate
            // P columns the softmax did not wait for the earlier ones; each S
            // MMA was issued only after the P V MMA before it had completed,
            // so those are complete already.
            if (!SEP) cpv += n_kv - lo - 1;
            if (!fa_wait_warp(&bar_pv[t], cpv & 1, 34 + t, wc)) { ok = false; break; }
            ++cpv;
            tc_fence_after();
            uint32_t ov[D / 32][32];
#pragma unroll
            for (int c0 = 0; c0 < D / 32; ++c0) tmem_ld32(lane_addr + col_o + c0 * 32, ov[c0]);
            tmem_ld_wait(ov[0]);
#pragma unroll
            for (int c0 = 1; c0 < D / 32; ++c0) asm volatile("" : FA_R32(ov[c0]) : : "memory");
            tc_fence_before();
            mbar_arrive(&bar_o_free[t]);
            // CROSS: where the rows go is read again, not held in registers through the
            // loop over the keys.
            FwdTile out = wt;
            int seg = -1;   // the segment's slot
            if constexpr (CROSS) {
                asm volatile("" ::: "memory");
                out = sch.tile();
                seg = sch.tile().slot;
            }
            const bool valid = row < out.len;
            // a row that sees no key (the exponentials of the FMA pipe are not quite 0);
            // scores of NaN, which the maximum passes over, leave l NaN
            if (CROSS && m2 == -CUDART_INF_F && l == l) {
                l = 0.0f;
#pragma unroll
                for (int c0 = 0; c0 < D / 32; ++c0)
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[c0][e] = 0u;
            }
            const float l_o = PRECISE ? l + lc : l;
            const float inv_l = (l_o > 0.0f) ? 1.0f / l_o : 0.0f;
            if (seg >= 0) {   // a segment: the join makes the rows of it
                if (valid) {
                    const int r = t * kBM + rl;
                    float4* dst = p.part_o + (size_t)seg * (D / 4) * (kTiles * kBM) + r;
#pragma unroll
                    for (int c0 = 0; c0 < D / 4; ++c0)
                        dst[c0 * (kTiles * kBM)] =
                            make_float4(__uint_as_float(ov[c0 / 8][c0 % 8 * 4 + 0]) * inv_l,
                                        __uint_as_float(ov[c0 / 8][c0 % 8 * 4 + 1]) * inv_l,
                                        __uint_as_float(ov[c0 / 8][c0 % 8 * 4 + 2]) * inv_l,
                                        __uint_as_float(ov[c0 / 8][c0 % 8 * 4 + 3]) * inv_l);
                    p.part_lse[(size_t)seg * (kTiles * kBM) + r] =
                        l == 0.0f ? -CUDART_INF_F : m2 + log2f(l);
                }
                continue;
            }
            const size_t orow = ((size_t)out.q_z * p.rows + out.tok0 + (valid ? row : 0)) * D;
            if (valid) {
#pragma unroll
                for (int c0 = 0; c0 < D / 32; ++c0) {
                    if (PRECISE) {
                        float4* dst =
                            reinterpret_cast<float4*>(static_cast<float*>(p.o) + orow + c0 * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 8; ++q4)
                            dst[q4] = make_float4(__uint_as_float(ov[c0][q4 * 4 + 0]) * inv_l,
                                                  __uint_as_float(ov[c0][q4 * 4 + 1]) * inv_l,
                                                  __uint_as_float(ov[c0][q4 * 4 + 2]) * inv_l,
                                                  __uint_as_float(ov[c0][q4 * 4 + 3]) * inv_l);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(
                            static_cast<__nv_bfloat16*>(p.o) + orow + c0 * 32);
#pragma unroll
                        for (int q4 = 0; q4 < 4; ++q4) {
                            uint4 w;
                            w.x = pack_bf16x2(__uint_as_float(ov[c0][q4 * 8 + 0]) * inv_l,
                                              __uint_as_float(ov[c0][q4 * 8 + 1]) * inv_l);
                            w.y = pack_bf16x2(__uint_as_float(ov[c0][q4 * 8 + 2]) * inv_l,
                                              __uint_as_float(ov[c0][q4 * 8 + 3]) * inv_l);
                            w.z = pack_bf16x2(__uint_as_float(ov[c0][q4 * 8 + 4]) * inv_l,
                                              __uint_as_float(ov[c0][q4 * 8 + 5]) * inv_l);
                            w.w = pack_bf16x2(__uint_as_float(ov[c0][q4 * 8 + 6]) * inv_l,
                                              __uint_as_float(ov[c0][q4 * 8 + 7]) * inv_l);
                            dst[q4] = w;
                        }
                    }
                }
                p.lse[(size_t)out.q_z * p.rows + out.tok0 + row] =
                    (CROSS ? l != 0.0f : l > 0.0f) ? (m2 + log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
            }
            if (p.lse_ext != nullptr && row0 < p.Np) {
                // Training forward: this tile's rows of the backward workspace
                // (a tile lies wholly below Np or wholly past it: both are
                // multiples of 128).  The -LSE row as the preprocess would
                // write it from the stored LSE (padding rows past N get -1e30,
                // so P = 0 there), and the tile's 128 fp32 dQ accumulator rows
                // zeroed, contiguous in memory: consecutive threads write
                // consecutive 16-byte pieces, so each warp store is coalesced.
                const long long r0 = (long long)wt.bh * p.Np + row0;
                const float lse_row =
                    (l > 0.0f) ? (m2 + log2f(l)) * 0.69314718055994531f : -CUDART_INF_F;
                write_lse_ext_row(p.lse_ext, r0 + rl,
                                  valid ? -lse_row * 1.4426950408889634f : -1e30f);
                float4* z = reinterpret_cast<float4*>(p.dq_acc + r0 * D);
#pragma unroll
                for (int c4 = 0; c4 < D / 4; ++c4) z[c4 * kBM + rl] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
        if (!PRECISE && warp == kProducerWarp && lane == 0) {
            // ------------------------------------------------- K producer
            tma_prefetch_desc(&tm_k);
            uint32_t g = 0;              // K blocks loaded so far (ring position)
            bool ok = true;
            if constexpr (CROSS) {
                // The next item goes into the ring once this one's first block is on its way.
                CrossWalk walk(share);
                uint32_t n = 0;   // items put into the ring
                CrossTile nxt;
                auto put = [&] {
                    const uint32_t r = n % kRing;
                    if (n >= (uint32_t)kRing && !fa_wait(&ring.empty[r], (n / kRing - 1) & 1, 41, wc))
                        return false;
                    nxt.n_kv[kTiles - 1] = 0;
                    if (walk.next(p, causal)) nxt = cross_tile(walk, p, causal);
                    ring.tile[r] = nxt;
                    mbar_arrive(&ring.full[r]);
                    ++n;
                    return true;
                };
                ok = put();
                while (ok && nxt.n_kv[kTiles - 1] > 0) {
                    const CrossTile wt = nxt;
                    for (int j = wt.lo[0]; j < wt.n_kv[kTiles - 1]; ++j, ++g) {
                        const int s = g % SK;
                        if (g >= (uint32_t)SK &&
                            !fa_wait(&bar_k_empty[s], ((g / SK) - 1) & 1, 10, wc)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bar_k[s], Cfg::kTileBytes);
                        for (int c = 0; c < Cfg::kChunks; ++c)
                            tma_load_3d(sK + s * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_k,
                                        &bar_k[s], c * 64, wt.ktok0 + j * kBN, wt.kv_z);
                        if (j == wt.lo[0]) ok = put();
                    }
                }
            } else {
                FwdSched<VARLEN, CROSS> sch = sched(false);
                for (int item = sch.next(p, causal); ok && item < p.n_items;
                     item = sch.next(p, causal)) {
                    const FwdTile wt = tile(item, sch);
                    for (int j = wt.lo[0]; j < wt.n_kv[kTiles - 1]; ++j, ++g) {
                        const int s = g % SK;
                        if (g >= (uint32_t)SK && !fa_wait(&bar_k_empty[s], ((g / SK) - 1) & 1, 10, wc)) {
                            ok = false;
                            break;
                        }
                        mbar_arrive_expect_tx(&bar_k[s], Cfg::kTileBytes);
                        for (int c = 0; c < Cfg::kChunks; ++c)
                            tma_load_3d(sK + s * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_k, &bar_k[s],
                                        c * 64, wt.ktok0 + j * kBN, wt.kv_z);
                    }
                }
            }
            if (abort_sh) {   // drain the copies still in flight (bounded)
                const WaitCtx dc{p.status, nullptr};
                for (uint32_t x = (g > (uint32_t)SK ? g - SK : 0); x < g; ++x)
                    fa_wait(&bar_k[x % SK], (x / SK) & 1, 11, dc);
            }
        } else if (!PRECISE && warp == kVProducerWarp && lane == 0) {
            // ---------------------------------------------- V and Q producer
            // The Q tiles of an item are loaded ahead of its V blocks, as soon
            // as the last S MMAs of the previous item have read the old ones.
            tma_prefetch_desc(&tm_v);
            tma_prefetch_desc(&tm_q);
            uint32_t g = 0;
            int lt = 0, q_loaded = -1;
            bool ok = true;
            FwdSched<VARLEN, CROSS> sch = sched(false);
            for (int item = sch.next(p, causal); ok && item < p.n_items;
                 item = sch.next(p, causal), ++lt) {
                const FwdTile wt = tile(item, sch);
                for (int t = 0; t < kTiles; ++t) {
                    if (lt > 0 && !fa_wait(&bar_q_free[t], (lt - 1) & 1, 12, wc)) { ok = false; break; }
                    mbar_arrive_expect_tx(&bar_q[t], Cfg::kTileBytes);
                    for (int c = 0; c < Cfg::kChunks; ++c)
                        tma_load_3d(sQ + t * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_q,
                                    &bar_q[t], c * 64, wt.tok0 + wt.row_base + t * kBM, wt.q_z);
                }
                if (!ok) break;
                q_loaded = lt;
                for (int j = wt.lo[0]; j < wt.n_kv[kTiles - 1]; ++j, ++g) {
                    const int s = g % SV;
                    if (g >= (uint32_t)SV && !fa_wait(&bar_v_empty[s], ((g / SV) - 1) & 1, 13, wc)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bar_v[s], Cfg::kTileBytes);
                    for (int c = 0; c < Cfg::kChunks; ++c)
                        tma_load_3d(sV + s * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_v, &bar_v[s],
                                    c * 64, wt.ktok0 + j * kBN, wt.kv_z);
                }
            }
            if (abort_sh) {   // drain the copies still in flight (bounded)
                const WaitCtx dc{p.status, nullptr};
                for (uint32_t x = (g > (uint32_t)SV ? g - SV : 0); x < g; ++x)
                    fa_wait(&bar_v[x % SV], (x / SV) & 1, 14, dc);
                if (q_loaded >= 0)
                    for (int t = 0; t < kTiles; ++t) fa_wait(&bar_q[t], q_loaded & 1, 15, dc);
            }
        } else if (warp == kProducerWarp && (PRECISE || lane == 0)) {
            // ------------------------------------- K producer, PRECISE form
            // (This and the next form are written to cover the bf16 case as
            // well, where the branches above take it first; equivalent to
            // PRECISE-only conditions, but the kernel built from this form
            // measured 8 % faster.)
            // The whole warp runs this loop (lane 0 issues the copies) and,
            // before issuing K_g, converts its half of V_{g-2}.
            // Issuing K_g waits for the S MMAs of K_{g-SK}, which follow the
            // P V MMAs of V_{g-SK-1}, whose half was converted before; the
            // issue of V_{g-2} waits for nothing this warp does from here on.
            const bool leader = (lane == 0);
            if (leader) tma_prefetch_desc(&tm_k);
            uint32_t g = 0, gc = 0;      // K blocks loaded (ring position); V halves converted
            bool ok = true;
            FwdSched<VARLEN, CROSS> sch = sched(false);
            for (int item = sch.next(p, causal); ok && item < p.n_items;
                 item = sch.next(p, causal)) {
                const FwdTile wt = tile(item, sch);
                for (int j = wt.lo[0]; j < wt.n_kv[kTiles - 1]; ++j, ++g) {
                    if (PRECISE && gc + 2 <= g) {
                        if (!convert_v_half<SV, Cfg::kTileBytes>(sV, bar_v, bar_v_cvt, gc, 1, lane, wc)) {
                            ok = false;
                            break;
                        }
                        ++gc;
                    }
                    const int s = g % SK;
                    if (g >= (uint32_t)SK && !(PRECISE ? fa_wait_warp(&bar_k_empty[s], ((g / SK) - 1) & 1, 10, wc)
                                                       : fa_wait(&bar_k_empty[s], ((g / SK) - 1) & 1, 10, wc))) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        mbar_arrive_expect_tx(&bar_k[s], Cfg::kTileBytes);
                        for (int c = 0; c < Cfg::kChunks; ++c)
                            tma_load_3d(sK + s * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_k,
                                        &bar_k[s], c * 64, wt.tok0 + j * kBN, wt.kv_z);
                    }
                }
            }
            while (PRECISE && ok && gc < g)
                ok = convert_v_half<SV, Cfg::kTileBytes>(sV, bar_v, bar_v_cvt, gc++, 1, lane, wc);
            if (abort_sh && leader) {   // drain the copies still in flight (bounded)
                const WaitCtx dc{p.status, nullptr};
                for (uint32_t x = (g > (uint32_t)SK ? g - SK : 0); x < g; ++x)
                    fa_wait(&bar_k[x % SK], (x / SK) & 1, 11, dc);
            }
        } else if (warp == kVProducerWarp && (PRECISE || lane == 0)) {
            // -------------------------------- V and Q producer, PRECISE form
            // The whole warp runs this loop (lane 0 issues the copies) and
            // re-encodes its half of each V_g as fp16 as soon as it has
            // landed, before issuing V_{g+1}; the P V issuer waits for that
            // and for the K producer warp's half.  Issuing V_{g+1} waits for
            // the P V MMAs of V_{g+1-SV}, converted before, so the two never
            // wait on each other.  An item's first V block is issued ahead of
            // its Q tiles, so that it lands while the Q loads wait for the
            // previous item's last S MMAs.
            const bool leader = (lane == 0);
            if (leader) {
                tma_prefetch_desc(&tm_v);
                tma_prefetch_desc(&tm_q);
            }
            uint32_t g = 0;   // V blocks issued (and their first halves converted)
            int lt = 0, q_loaded = -1;
            bool ok = true;
            FwdSched<VARLEN, CROSS> sch = sched(false);
            for (int item = sch.next(p, causal); ok && item < p.n_items;
                 item = sch.next(p, causal), ++lt) {
                const FwdTile wt = tile(item, sch);
                const int jb = wt.lo[0], je = wt.n_kv[kTiles - 1];
                auto issue_v = [&](int j) -> bool {   // V_j into the ring
                    const int s = g % SV;
                    if (g >= (uint32_t)SV && !(PRECISE ? fa_wait_warp(&bar_v_empty[s], ((g / SV) - 1) & 1, 13, wc) : fa_wait(&bar_v_empty[s], ((g / SV) - 1) & 1, 13, wc)))
                        return false;
                    if (leader) {
                        mbar_arrive_expect_tx(&bar_v[s], Cfg::kTileBytes);
                        for (int c = 0; c < Cfg::kChunks; ++c)
                            tma_load_3d(sV + s * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_v,
                                        &bar_v[s], c * 64, wt.tok0 + j * kBN, wt.kv_z);
                    }
                    ++g;
                    return true;
                };
                const bool pre = PRECISE && jb < je;
                if (pre && !issue_v(jb)) { ok = false; break; }
                for (int t = 0; t < kTiles; ++t) {
                    if (lt > 0 && !(PRECISE ? fa_wait_warp(&bar_q_free[t], (lt - 1) & 1, 12, wc) : fa_wait(&bar_q_free[t], (lt - 1) & 1, 12, wc))) { ok = false; break; }
                    if (leader) {
                        mbar_arrive_expect_tx(&bar_q[t], Cfg::kTileBytes);
                        for (int c = 0; c < Cfg::kChunks; ++c)
                            tma_load_3d(sQ + t * Cfg::kTileBytes + c * Cfg::kChunkBytes, &tm_q,
                                        &bar_q[t], c * 64, wt.tok0 + wt.row_base + t * kBM, wt.q_z);
                    }
                }
                if (!ok) break;
                q_loaded = lt;
                for (int j = jb; j < je; ++j) {
                    // (issue_v counts V_j before the conversion: an abort drains it)
                    if (!(pre && j == jb) && !issue_v(j)) { ok = false; break; }
                    if (PRECISE && !convert_v_half<SV, Cfg::kTileBytes>(sV, bar_v, bar_v_cvt, g - 1, 0, lane, wc)) {
                        ok = false;
                        break;
                    }
                }
            }
            if (abort_sh && leader) {   // drain the copies still in flight (bounded)
                const WaitCtx dc{p.status, nullptr};
                for (uint32_t x = (g > (uint32_t)SV ? g - SV : 0); x < g; ++x)
                    fa_wait(&bar_v[x % SV], (x / SV) & 1, 14, dc);
                if (q_loaded >= 0)
                    for (int t = 0; t < kTiles; ++t) fa_wait(&bar_q[t], q_loaded & 1, 15, dc);
            }
        } else if (warp == kPvWarp && lane == 0) {
            // ------------------------------------------- P V MMA issuer
            // O_t += P_t V_j, P_t read from TMEM.  A second issuing thread:
            // while the S issuer waits or commits, this one keeps the tensor
            // core busy, and the other way round.
            constexpr uint32_t idesc_o =
                PRECISE ? idesc_f16_f32(kBM, D, false, true) : idesc_bf16_f32(kBM, D, false, true);
            const uint32_t sv = smem_u32(sV);
            uint32_t g = 0, cp0 = 0, cp1 = 0;       // V blocks used; P_t arrivals seen
            bool ok = true;
            int lt = 0;
            auto pv = [&](auto tc, uint32_t vstage, bool first, bool wait_o) -> bool {
                constexpr int T = decltype(tc)::value;
                constexpr uint32_t col_o = T ? Cfg::kColO1 : Cfg::kColO0;
                constexpr uint32_t col_s = T ? Cfg::kColS1 : Cfg::kColS0;
                constexpr uint32_t col_p = SEP ? (T ? Cfg::kColP1 : Cfg::kColP0) : col_s;
                uint32_t& c = T ? cp1 : cp0;
                if (!fa_wait(&bar_p[T], c & 1, 24 + T, wc)) return false;
                ++c;
                if (wait_o && !fa_wait(&bar_o_free[T], (lt - 1) & 1, 26 + T, wc)) return false;
                tc_fence_after();
                const uint64_t vd = sdesc_sw128(sv + vstage * Cfg::kTileBytes, Cfg::kChunkBytes, 1024);
#pragma unroll
                for (int kk = 0; kk < kBN / 16; ++kk)
                    mma_ts(tmem + col_o, tmem + col_p + kk * 8, vd + mnmajor_step(kk), idesc_o,
                           (!first || kk > 0) ? 1u : 0u);
                mma_commit(&bar_pv[T]);
                return true;
            };
            FwdSched<VARLEN, CROSS> sch = sched(false);
            for (int item = sch.next(p, causal); ok && item < p.n_items;
                 item = sch.next(p, causal), ++lt) {
                const FwdTile wt = tile(item, sch);
                // Key blocks [lo0, n0) for tile 0, [lo1, n1) for tile 1, with
                // lo0 <= lo1 and n0 <= n1; V_j streams for j in [lo0, n1).
                const int lo0 = wt.lo[0], lo1 = wt.lo[1], n0 = wt.n_kv[0], n1 = wt.n_kv[1];
                for (int j = lo0; j < n1; ++j) {
                    const uint32_t gj = g + (j - lo0), vs = gj % SV;
                    // V_j landed (PRECISE: and re-encoded as fp16)
                    if (!fa_wait(PRECISE ? &bar_v_cvt[vs] : &bar_v[vs], (gj / SV) & 1, 22, wc)) {
                        ok = false;
                        break;
                    }
                    if (j < n0 && !pv(std::integral_constant<int, 0>{}, vs, j == lo0,
                                      j == lo0 && lt > 0)) {
                        ok = false;
                        break;
                    }
                    if (j >= lo1 && !pv(std::integral_constant<int, 1>{}, vs, j == lo1,
                                        j == lo1 && lt > 0)) {
                        ok = false;
                        break;
                    }
                    mma_commit(&bar_v_empty[vs]);            // V_j read by both PVs
                }
                g += n1 - lo0;
            }
            if constexpr (CROSS) ok = ok && sch.ok;
            if (!ok) {   // no MMA of this thread may still write TMEM at teardown
                __shared__ uint64_t bar_drain_pv;
                mbar_init(&bar_drain_pv, 1);
                fence_mbar_init();
                mma_commit(&bar_drain_pv);
                fa_wait(&bar_drain_pv, 0, 29, WaitCtx{p.status, nullptr});
            }
        } else if (warp == kMmaWarp && lane == 0) {
            // ---------------------------------------------- S MMA issuer
            // S_t(j) = Q_t K_j^T goes out as soon as K_j has landed and the
            // columns of S_t are free again: loaded by the softmax (P in
            // columns of its own), or read by the P_t V MMA of the previous
            // block (P written over S).  The tile index is a compile-time
            // constant in every MMA, so operand addresses fold into the
            // instruction stream.
            constexpr uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, false, false);
            const uint32_t sq = smem_u32(sQ), sk = smem_u32(sK);
            uint32_t g = 0, ns0 = 0, ns1 = 0;       // K blocks used; S_t MMAs issued
            bool ok = true;
            int lt = 0;
            auto s_mma = [&](auto tc, uint32_t kstage) -> bool {
                constexpr int T = decltype(tc)::value;
                uint32_t& n = T ? ns1 : ns0;
                if (n > 0 && !fa_wait(SEP ? &bar_s_free[T] : &bar_pv[T], (n - 1) & 1, 36 + T, wc))
                    return false;
                ++n;
                tc_fence_after();
                const uint64_t qd = sdesc_sw128(sq + T * Cfg::kTileBytes, 16, 1024);
                const uint64_t kd = sdesc_sw128(sk + kstage * Cfg::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + (T ? Cfg::kColS1 : Cfg::kColS0),
                           qd + kmajor_step(kk, Cfg::kChunkBytes),
                           kd + kmajor_step(kk, Cfg::kChunkBytes), idesc_s, kk > 0);
                mma_commit(&bar_s[T]);
                return true;
            };
            FwdSched<VARLEN, CROSS> sch = sched(false);
            for (int item = sch.next(p, causal); ok && item < p.n_items;
                 item = sch.next(p, causal), ++lt) {
                const FwdTile wt = tile(item, sch);
                const int lo0 = wt.lo[0], lo1 = wt.lo[1], n0 = wt.n_kv[0], n1 = wt.n_kv[1];
                if (!fa_wait(&bar_q[0], lt & 1, 20, wc) || !fa_wait(&bar_q[1], lt & 1, 20, wc)) {
                    ok = false;
                    break;
                }
                for (int j = lo0; j < n1; ++j) {
                    const uint32_t gj = g + (j - lo0), ks = gj % SK;
                    if (!fa_wait(&bar_k[ks], (gj / SK) & 1, 21, wc)) { ok = false; break; }
                    if (j < n0) {
                        if (!s_mma(std::integral_constant<int, 0>{}, ks)) { ok = false; break; }
                        if (j + 1 == n0) mma_commit(&bar_q_free[0]);
                    }
                    if (j >= lo1) {
                        if (!s_mma(std::integral_constant<int, 1>{}, ks)) { ok = false; break; }
                        if (j + 1 == n1) mma_commit(&bar_q_free[1]);
                    }
                    mma_commit(&bar_k_empty[ks]);            // K_j read by both S MMAs
                }
                g += n1 - lo0;
            }
            if constexpr (CROSS) ok = ok && sch.ok;
            if (!ok) {
                __shared__ uint64_t bar_drain;
                mbar_init(&bar_drain, 1);
                fence_mbar_init();
                mma_commit(&bar_drain);
                fa_wait(&bar_drain, 0, 29, WaitCtx{p.status, nullptr});
            }
        }
        __syncwarp();
    }

    if (CROSS && threadIdx.x == 0 && p.split) p.part_at[blockIdx.x] = share[0];
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The items that went to several CTAs: O = sum over the segments of 2^(L_s - L) O_s with
// L = log2 sum 2^L_s, L_s the segment's LSE.  Block (c, y) has the item in whose middle
// CTA c's share begins, if c is the first such, and 16 columns of O; one row a thread.
// Bound by the reads of the segments (from L2: they were just written).
template <int D>
__global__ void __launch_bounds__(kTiles * kBM)
cross_join_kernel(const FwdParams p, int ctas) {
    pdl_wait();
    const int c = blockIdx.x + 1, r = threadIdx.x;
    const CrossAt at = p.part_at[c], prev = p.part_at[c - 1];
    if (at.blk == 0 || (prev.b == at.b && prev.it == at.it && prev.blk > 0)) return;
    const CrossSeq sq(p, at.b, p.causal);
    const int G = p.H / p.Hkv;
    const int h = at.it / G / sq.M * G + at.it % G;
    const int row = at.it / G % sq.M * (kTiles * kBM) + r;
    if (row >= sq.len) return;
    int last = c;
    while (last + 1 < ctas) {
        const CrossAt a = p.part_at[last + 1];
        if (a.b != at.b || a.it != at.it || a.blk == 0) break;
        ++last;
    }
    auto slot = [&](int x) { return (size_t)(2 * x + (x < c ? 1 : 0)); };
    float top = -CUDART_INF_F;
    for (int x = c - 1; x <= last; ++x) top = fmaxf(top, p.part_lse[slot(x) * (kTiles * kBM) + r]);
    const float m = top == -CUDART_INF_F ? 0.0f : top;
    float sum = 0.0f, acc[16] = {};
#pragma unroll 2
    for (int x = c - 1; x <= last; ++x) {
        const float w = ex2(p.part_lse[slot(x) * (kTiles * kBM) + r] - m);
        const float4* src =
            p.part_o + (slot(x) * (D / 4) + blockIdx.y * 4) * (kTiles * kBM) + r;
        sum += w;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 v = src[u * (kTiles * kBM)];
            acc[4 * u + 0] = fmaf(w, v.x, acc[4 * u + 0]);
            acc[4 * u + 1] = fmaf(w, v.y, acc[4 * u + 1]);
            acc[4 * u + 2] = fmaf(w, v.z, acc[4 * u + 2]);
            acc[4 * u + 3] = fmaf(w, v.w, acc[4 * u + 3]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const size_t z = p.cu_seqlens ? (size_t)h : (size_t)at.b * p.H + h;
    const size_t orow = z * p.rows + sq.tok0 + row;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + orow * D +
                                          blockIdx.y * 16);
#pragma unroll
    for (int u = 0; u < 2; ++u)
        dst[u] = make_uint4(pack_bf16x2(acc[8 * u + 0] * inv, acc[8 * u + 1] * inv),
                            pack_bf16x2(acc[8 * u + 2] * inv, acc[8 * u + 3] * inv),
                            pack_bf16x2(acc[8 * u + 4] * inv, acc[8 * u + 5] * inv),
                            pack_bf16x2(acc[8 * u + 6] * inv, acc[8 * u + 7] * inv));
    if (blockIdx.y == 0)
        p.lse[orow] =
            sum == 0.0f ? -CUDART_INF_F : (m + log2f(sum)) * 0.69314718055994531f;
}

template <int D, bool CAUSAL, bool PRECISE, bool WINDOW = false, bool VARLEN = false,
          bool CROSS = false>
cudaError_t launch_fwd_t(const Shape& s, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const FwdParams& p, int grid,
                         cudaStream_t stream) {
    auto kern = fa_fwd_kernel<D, CAUSAL, PRECISE, WINDOW, VARLEN, CROSS>;
    static int configured_device = -1;   // attribute is per device; cheap to repeat
    int dev = 0;
    cudaGetDevice(&dev);
    if (configured_device != dev) {
        // The register split must fit in what the launch provides, or the
        // setmaxnreg.inc of the softmax warps would wait forever.
        cudaFuncAttributes attr;
        cudaError_t e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return e;
        if (attr.numRegs * kThreads < kRegsNeeded) return cudaErrorInvalidConfiguration;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 FwdCfg<D, PRECISE>::kSmemAlloc);
        if (e != cudaSuccess) return e;
        configured_device = dev;
    }
    kern<<<grid, kThreads, FwdCfg<D, PRECISE>::kSmemAlloc, stream>>>(tq, tk, tv, p);
    return cudaGetLastError();
}

}  // namespace

// Keys of another length: the most CTAs that a split call has.
static long long split_ctas(const Shape& s) {
    const long long items = (long long)s.B * s.H * ((s.N + kTiles * kBM - 1) / (kTiles * kBM));
    const long long n = (s.Nk + kBN - 1) / kBN;
    return n <= kSplitBlocks ? 0 : std::min<long long>(kMaxCtas, (items * n + kMinBlocks - 1) / kMinBlocks);
}

size_t cross_fwd_workspace_bytes(const Shape& s) {
    return std::max<size_t>(
        256, split_ctas(s) * (2 * (kTiles * kBM) * (s.d + 1) * sizeof(float) + sizeof(CrossAt)));
}

// CTAs, and are there segments?  Only where an even share and the join are shorter than
// the rounds of whole items; from what the host knows, the sizes (padded sequences
// counted in full, packed ones as equally long).
static int cross_ctas(const Shape& s, bool& split) {
    const int sms = std::min(device_sm_count() > 0 ? device_sm_count() : 148, kMaxCtas);
    const long long rows = s.cu_seqlens ? s.total / s.B : s.N;
    const long long keys = s.cu_k ? std::min(s.total_k / s.B, s.Nk) : s.Nk;
    const long long M = std::max(1ll, (rows + kTiles * kBM - 1) / (kTiles * kBM));
    const long long n = (keys + kBN - 1) / kBN, q = (s.Nk - s.N) / kBN;
    double blocks = 0.0;   // of the pairs of one head
    for (long long m = 0; m < M; ++m)
        blocks += kItemCost + (s.causal ? std::min(std::max(2 * (m + 1) + q, 1ll), n) : n);
    const double items = (double)s.B * s.H * M, share = (double)s.B * s.H * blocks / sms;
    const double longest = (s.Nk + kBN - 1) / kBN + kItemCost;
    const double whole = std::max(longest, std::ceil(items / sms) * blocks / M);
    split = split_ctas(s) > 0 && std::max(share, (double)kMinBlocks) + kJoinCost < whole;
    const long long most = (long long)s.B * s.H * ((s.N + kTiles * kBM - 1) / (kTiles * kBM));
    return (int)std::min<long long>(sms, split ? split_ctas(s) : most);
}

static cudaError_t launch_fwd_cross(const Shape& s, const CUtensorMap& tq, const CUtensorMap& tk,
                                    const CUtensorMap& tv, FwdParams p, void* workspace,
                                    cudaStream_t stream) {
    bool split;
    const int ctas = cross_ctas(s, split);
    p.split = split;
    p.part_o = static_cast<float4*>(workspace);
    p.part_lse = static_cast<float*>(workspace) + (size_t)2 * ctas * (kTiles * kBM) * s.d;
    p.part_at = reinterpret_cast<CrossAt*>(p.part_lse + (size_t)2 * ctas * (kTiles * kBM));
    cudaError_t e =
        s.d == 128
            ? launch_fwd_t<128, false, false, false, false, true>(s, tq, tk, tv, p, ctas, stream)
            : launch_fwd_t<64, false, false, false, false, true>(s, tq, tk, tv, p, ctas, stream);
    if (e != cudaSuccess || !split || ctas < 2) return e;
    const dim3 grid(ctas - 1, s.d / 16);
    return s.d == 128 ? launch_pdl(cross_join_kernel<128>, grid, kTiles * kBM, 0, 1, stream, p, ctas)
                      : launch_pdl(cross_join_kernel<64>, grid, kTiles * kBM, 0, 1, stream, p, ctas);
}

cudaError_t launch_fwd(const Shape& s, const void* q, const void* k, const void* v, void* o,
                       float* lse, bool precise, DeviceStatus* status, cudaStream_t stream,
                       const BwdWorkspace* train_ws, void* cross_ws) {
    // Dense: maps {d, N, B*H(kv)}.  Packed variable lengths: {d, total, H(kv)},
    // a sequence's rows addressed from its first row.
    const bool varlen = s.cu_seqlens != nullptr, cross = s.Nk > 0;
    const int rows = varlen ? s.total : s.N;
    const int krows = !cross ? rows : varlen ? s.total_k : s.Nk;
    CUtensorMap tq, tk, tv;
    if (!make_tmap_bf16_3d(&tq, q, s.d, rows, varlen ? s.H : s.B * s.H, kBM) ||
        !make_tmap_bf16_3d(&tk, k, s.d, krows, varlen ? s.Hkv : s.B * s.Hkv, kBN) ||
        !make_tmap_bf16_3d(&tv, v, s.d, krows, varlen ? s.Hkv : s.B * s.Hkv, kBN))
        return cudaErrorInvalidValue;
    FwdParams p;
    p.Nk = s.Nk;
    p.krows = krows;
    p.kv_lens = s.kv_lens;
    p.cu_k = s.cu_k;
    p.H = s.H;
    p.Hkv = s.Hkv;
    p.N = s.N;
    p.rows = rows;
    p.cu_seqlens = s.cu_seqlens;
    p.BH = s.B * s.H;
    p.n_mblk = (s.N + kTiles * kBM - 1) / (kTiles * kBM);
    p.n_items = p.n_mblk * p.BH;
    p.causal = s.causal;
    p.window = s.window > 0 ? s.window : kNoWindow;
    p.scale_log2 = (float)((double)s.scale * 1.4426950408889634);
    p.o = o;
    p.lse = lse;
    p.status = status;
    p.lse_ext = nullptr;
    p.dq_acc = nullptr;
    p.Np = padded_rows(s.N);
    if (train_ws) {   // dense batches only (packed ones keep the plain preprocess)
        if (varlen) return cudaErrorInvalidValue;
        p.lse_ext = train_ws->lse_ext;
        p.dq_acc = train_ws->dq_acc;
    }
    // Persistent: one CTA per SM (at most one work item per CTA when there
    // are fewer items than SMs).
    const int sms = device_sm_count() > 0 ? device_sm_count() : 148;
    const int grid = p.n_items < sms ? p.n_items : sms;
    count_launch();
    const bool c = s.causal != 0;
    if (cross) {   // keys of another length (bf16 output, no window, no training form)
        if (precise || s.window > 0 || train_ws) return cudaErrorInvalidValue;
        return launch_fwd_cross(s, tq, tk, tv, p, cross_ws, stream);
    }
    if (varlen) {   // packed variable-length sequences (bf16 output, no window)
        if (precise || s.window > 0) return cudaErrorInvalidValue;
        if (s.d == 128)
            return c ? launch_fwd_t<128, true, false, false, true>(s, tq, tk, tv, p, grid, stream)
                     : launch_fwd_t<128, false, false, false, true>(s, tq, tk, tv, p, grid, stream);
        return c ? launch_fwd_t<64, true, false, false, true>(s, tq, tk, tv, p, grid, stream)
                 : launch_fwd_t<64, false, false, false, true>(s, tq, tk, tv, p, grid, stream);
    }
    if (s.window > 0) {   // the causal sliding window (bf16 output only)
        if (!c || precise) return cudaErrorInvalidValue;
        return s.d == 128 ? launch_fwd_t<128, true, false, true>(s, tq, tk, tv, p, grid, stream)
                          : launch_fwd_t<64, true, false, true>(s, tq, tk, tv, p, grid, stream);
    }
    if (s.d == 128) {
        if (precise)
            return c ? launch_fwd_t<128, true, true>(s, tq, tk, tv, p, grid, stream)
                     : launch_fwd_t<128, false, true>(s, tq, tk, tv, p, grid, stream);
        return c ? launch_fwd_t<128, true, false>(s, tq, tk, tv, p, grid, stream)
                 : launch_fwd_t<128, false, false>(s, tq, tk, tv, p, grid, stream);
    }
    if (precise)
        return c ? launch_fwd_t<64, true, true>(s, tq, tk, tv, p, grid, stream)
                 : launch_fwd_t<64, false, true>(s, tq, tk, tv, p, grid, stream);
    return c ? launch_fwd_t<64, true, false>(s, tq, tk, tv, p, grid, stream)
             : launch_fwd_t<64, false, false>(s, tq, tk, tv, p, grid, stream);
}

}  // namespace fa
