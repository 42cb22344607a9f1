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
// shared memory (N is 16 to 64 columns), each of the 128 softmax threads owns
// one key and R scores, nothing is computed for absent query rows past the next
// 8, 16 or 32, and no thread needs another's score: the running maximum m of a
// row moves only when some key passes it by 2^kSlack (a vote of the four
// warps), the row sums stay one partial per thread until the end, and the
// rescale of O^T touches kN columns.
//
// e4m3 pages are multiplied as they are.  A bf16 query row, times the power of
// two that brings its largest entry into [2^7, 2^8), is the sum of two e4m3
// numbers (8 significant bits = 4 + 4, exact down to e4m3's smallest step, 2^-9), so
// B holds the rows' first terms and, RP columns on, their second terms, and
// the two scores are added in fp32.  K's scale is the softmax thread's own
// (one thread, one key).  V's scale vs goes into P: w = 2^(x - m) vs kPScale with
// m the running maximum of x + log2 vs, so that w <= 448, as two e4m3 terms
// again; a row of zeros has scale 0 and weighs nothing.  No pass converts the
// pages, and shared memory sees each of their bytes twice.
//
// Work: the tiles of all (sequence, kv head) pairs, in order, are one list of T
// that the CTAs share evenly (CTA c of n takes tiles c T / n .. (c + 1) T / n),
// found on the device from the lengths, so that ragged batches stay balanced and
// a captured graph replays with other lengths.  A pair that one CTA holds whole
// is finished there.  The others leave O / l and LSE of their part in slot c + i
// (i the pair's index: along the list either c or i grows, so slots are unique),
// and the combine kernel joins a pair's slots in order.
//
// Warps: 0-3 softmax, 4 loads K, V and scales (a lane a page), 5 issues MMAs, 6
// lays out the next pair's queries.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <atomic>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kTile = 128;              // keys per tile
constexpr int kThreads = 224;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kMinLogScale = -60.0f;  // V scales below 2^-60 no longer move the reference
constexpr int kSoftBar = 1;             // named barrier of the softmax warps

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
    int ctas;                           // of the split kernel
    float scale_log2;
    DeviceStatus* status;
};

// Sizes of one variant: head dimension, page type, query rows rounded up.
template <int D, bool F8, int RP>
struct Cfg {
    static constexpr int kN = F8 ? 2 * RP : (RP < 16 ? 16 : RP);   // MMA columns
    static constexpr int kRowBytes = F8 ? D : 2 * D;
    static constexpr int kSw = kRowBytes < 128 ? 64 : 128;         // swizzle = chunk width
    static constexpr int kChunks = kRowBytes / kSw;
    static constexpr int kTileBytes = kTile * kRowBytes;
    static constexpr int kQBytes = kN * kRowBytes;
    static constexpr int kPRow = F8 ? kTile : 2 * kTile;
    static constexpr int kPBytes = kN * kPRow;
    static constexpr int kScaleBytes = F8 ? 2 * kTile * 4 : 0;
    // d = 128 fills an SM with one CTA; d = 64 runs two, so that one's
    // softmax and epilogue hide behind the other's loads.
    static constexpr int kCtas = (D == 64 && RP <= 16) ? 2 : 1;
    static constexpr int kRing = (kCtas == 2 ? 96 : 192) * 1024;
    static constexpr int kStages =
        (kRing - (F8 && RP == 32 ? 16 * 1024 : 0)) / (2 * kTileBytes + kScaleBytes);
    static constexpr int kSmem =
        kStages * (2 * kTileBytes + kScaleBytes) + 2 * kQBytes + 2 * kPBytes + 1024;
    static constexpr int kTmemCols = 3 * kN <= 64 ? 64 : (3 * kN <= 128 ? 128 : 256);
    // How far a score may pass the running maximum before O is rescaled (log2):
    // bf16 P keeps its precision at any magnitude; e4m3 P ends at 448.
    static constexpr float kSlack = F8 ? 2.0f : 8.0f;
    static constexpr float kPScale = F8 ? 112.0f : 1.0f;           // 2^kSlack * kPScale = 448
};

__device__ __forceinline__ int clamped_len(const PagedParams& p, int b) {
    return min(max(__ldg(p.seqlens + b), 0), p.max_pages << p.ps_shift);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// A CTA's place in the list of tiles: pair (b, g), tile t of it, and how many
// tiles the CTA still has.
struct Cursor {
    int b, g, len, t, left;
    // tiles of the current pair that belong to this CTA
    __device__ __forceinline__ int run() const { return min(tiles_of(len) - t, left); }
    // past `n` tiles of the current pair
    __device__ __forceinline__ void skip(const PagedParams& p, int n) {
        left -= n;
        t += n;
        if (left > 0 && t == tiles_of(len)) {
            t = 0;
            if (++g == p.Hkv) {
                g = 0;
                // left > 0: a sequence with keys follows (the bound is for
                // lengths that somebody changes under the kernel)
                do {
                    if (++b >= p.B) {
                        left = 0;
                        return;
                    }
                    len = clamped_len(p, b);
                } while (len == 0);
            }
        }
    }
};

// Length of the list of tiles (returned) and the tiles of the sequences before
// lane's first and up to its last one: a warp adds up B lengths, each lane
// those of ceil(B / 32) neighbouring sequences b0 .. b1 - 1.
__device__ __forceinline__ int list_length(const PagedParams& p, int lane, int& b0, int& b1,
                                           int& before, int& upto) {
    const int per = (p.B + 31) / 32;
    b0 = min(p.B, lane * per);
    b1 = min(p.B, b0 + per);
    int mine = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) mine += tiles_of(clamped_len(p, b));
    mine *= p.Hkv;
    upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += y;
    }
    before = upto - mine;
    return __shfl_sync(0xffffffffu, upto, 31);
}

// CTA c of nc holds tiles c T / nc .. (c + 1) T / nc - 1; the one that holds
// tile t.  nc <= T, so that each one holds some and a pair's CTAs are neighbours.
__device__ __forceinline__ int cta_of_tile(int t, int T, int nc) {
    return (int)((((long long)t + 1) * nc + T - 1) / T) - 1;
}

// Monotone map of a float's order onto signed integers (its own inverse).
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int i) {
    return __int_as_float(i ^ ((i >> 31) & 0x7fffffff));
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

template <int D, bool F8, int RP>
__global__ void __launch_bounds__(kThreads, (Cfg<D, F8, RP>::kCtas))
fa_decode_paged_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
    using C = Cfg<D, F8, RP>;
    constexpr int S = C::kStages, N = C::kN, TB = C::kTileBytes;
    constexpr uint32_t kColO = 2 * N;             // S buffers at 0 and N
    extern __shared__ uint8_t dsm_raw[];
    uint8_t* dsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsm_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    // Stage s: V, then K.  At d = 64 the MMA's 128 rows reach past V's 64
    // columns: its second half reads K, into rows of O^T that nobody reads.
    uint8_t* sKV = dsm;
    uint8_t* sQ = sKV + S * 2 * TB;               // [2]
    uint8_t* sP = sQ + 2 * C::kQBytes;            // [2]
    float* sScale = reinterpret_cast<float*>(sP + 2 * C::kPBytes);   // [S][segment][K, V][rows]
    __shared__ uint64_t bar_q[2], bar_q_free[2], bar_k[S], bar_k_empty[S], bar_v[S],
        bar_v_empty[S];
    // S_t, P_t and P_t V_t signal barrier t & 1 (t counts the CTA's tiles)
    __shared__ uint64_t bar_s[2], bar_p[2], bar_pv[2], bar_drain;
    __shared__ float4 row_part4[RP];              // [4 warps][RP]: maxima, then sums
    __shared__ float q_scale[2][RP];              // e4m3: score of one code product, log2 units
    __shared__ int row_query[RP];                 // r % Nq
    __shared__ int start_sh[4];                   // first pair and tile, tiles of this CTA
    __shared__ uint32_t tmem_base_sh;
    __shared__ int abort_sh;
    float* row_part = reinterpret_cast<float*>(row_part4);
    const WaitCtx wc{p.status, &abort_sh};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_launch_dependents();
    if (warp == 0) {
        int b0, b1, at, upto;
        const int T = list_length(p, lane, b0, b1, at, upto);
        const int nc = min((int)gridDim.x, T), c = min((int)blockIdx.x, nc);
        const int begin = nc ? (int)((long long)c * T / nc) : 0;
        const int end = c < nc ? (int)((long long)(c + 1) * T / nc) : begin;
        if (lane == 0 && begin == end) start_sh[3] = 0;
        if (begin < end && at <= begin && begin < upto) {
            for (int b = b0; b < b1; ++b) {
                const int tiles = tiles_of(clamped_len(p, b));
                if (begin < at + tiles * p.Hkv) {
                    start_sh[0] = b;
                    start_sh[1] = (begin - at) / tiles;
                    start_sh[2] = (begin - at) % tiles;
                    start_sh[3] = end - begin;
                    break;
                }
                at += tiles * p.Hkv;
            }
        }
    } else if (warp == 4) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
            abort_sh = 0;
            for (int x = 0; x < 2; ++x) {
                mbar_init(&bar_q[x], 32);
                mbar_init(&bar_q_free[x], F8 ? 5 : 1);   // the last S MMA; the warps' scales
                mbar_init(&bar_s[x], 1);
                mbar_init(&bar_p[x], 128);
                mbar_init(&bar_pv[x], 1);
            }
            for (int s = 0; s < S; ++s) {
                mbar_init(&bar_k[s], 1);
                mbar_init(&bar_k_empty[s], 1);
                mbar_init(&bar_v[s], 1);
                mbar_init(&bar_v_empty[s], 1);
            }
            mbar_init(&bar_drain, 1);
            fence_mbar_init();
        }
    } else if (warp == 5) {
        tmem_alloc(&tmem_base_sh, C::kTmemCols);
        tmem_relinquish();
    } else {
        // Query rows past R and columns of P past RP stay zero.
        const int x0 = (warp == 6 ? 3 : warp - 1) * 32 + lane;
        for (int e = x0; e < (2 * C::kQBytes + 2 * C::kPBytes) / 16; e += 128)
            reinterpret_cast<uint4*>(sQ)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (warp == 6)
            for (int r = lane; r < RP; r += 32) row_query[r] = r % p.Nq;
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    Cursor cur{start_sh[0], start_sh[1], 0, start_sh[2], start_sh[3]};
    if (cur.left > 0) cur.len = clamped_len(p, cur.b);

    if (warp == 4) {
        // ------------------------------------------------------- loads
        // Lanes 0-15 load K, 16-31 V, one box of up to 128 keys of one page
        // each; in e4m3 lanes 24-31 load the pages' scales instead.
        const int seg_shift = min(p.ps_shift, 7), seg = 1 << seg_shift;
        const int n_seg = kTile >> seg_shift;
        const bool is_scale = F8 && lane >= 24;
        const int x = is_scale ? lane - 24 : lane & 15;
        const int my_seg = is_scale ? x : x / C::kChunks, chunk = is_scale ? 0 : x % C::kChunks;
        const int seg_bytes = seg * C::kSw;
        auto page_of = [&](const Cursor& c) {
            const int key = c.t * kTile + my_seg * seg;
            return (my_seg < n_seg && key < c.len)
                       ? __ldg(p.table + (long long)c.b * p.max_pages + (key >> p.ps_shift))
                       : 0;
        };
        bool ok = true;
        int gt = 0, vt = 0;                       // K and V tiles loaded so far
        int page = cur.left > 0 ? page_of(cur) : 0;
        while (ok && cur.left > 0) {
            const Cursor at = cur;
            cur.skip(p, 1);
            const int page_next = cur.left > 0 ? page_of(cur) : 0;   // in flight during the waits
            const int s = gt % S;
            const int have = min(n_seg, (at.len - at.t * kTile + seg - 1) >> seg_shift);
            const bool mine = my_seg < have;
            const int key = at.t * kTile + my_seg * seg;
            const int row = key & ((1 << p.ps_shift) - 1);
            const bool known = (unsigned)page < (unsigned)p.n_pages;
            // a page outside the pool reads as zeros (past the map's last row)
            const int outer = (known ? page : p.n_pages) * p.Hkv + (known ? at.g : 0);
            uint8_t* stage = sKV + s * 2 * TB;
            if (gt >= S) ok = fa_wait_warp(&bar_k_empty[s], ((gt / S) - 1) & 1, 100, wc);
            if (ok) {
                if (lane == 0) mbar_arrive_expect_tx(&bar_k[s], have * seg_bytes * C::kChunks);
                __syncwarp();
                if (lane < 16 && mine)
                    tma_load_3d(stage + TB + chunk * (kTile * C::kSw) + my_seg * seg_bytes, &tm_k,
                                &bar_k[s], chunk * (F8 ? C::kSw : C::kSw / 2), row, outer);
                ++gt;
            }
            if (ok && vt >= S) ok = fa_wait_warp(&bar_v_empty[s], ((vt / S) - 1) & 1, 101, wc);
            if (ok) {
                if (lane == 0)
                    mbar_arrive_expect_tx(&bar_v[s],
                                          have * (seg_bytes * C::kChunks + (F8 ? 8 * seg : 0)));
                __syncwarp();
                if (lane >= 16 && mine && !is_scale)
                    tma_load_3d(stage + chunk * (kTile * C::kSw) + my_seg * seg_bytes, &tm_v,
                                &bar_v[s], chunk * (F8 ? C::kSw : C::kSw / 2), row, outer);
                if (is_scale && mine) {
                    const float* src =
                        p.scales + (((long long)(known ? page : 0) * p.Hkv + at.g) << (p.ps_shift + 1)) +
                        row;
                    float* dst = sScale + s * 2 * kTile + my_seg * 2 * seg;
                    if (p.ps_shift <= 7) {
                        bulk_load(dst, src, 8 * seg, &bar_v[s]);      // K's, then V's
                    } else {
                        bulk_load(dst, src, 4 * seg, &bar_v[s]);
                        bulk_load(dst + seg, src + (1 << p.ps_shift), 4 * seg, &bar_v[s]);
                    }
                }
            }
            if (ok) ++vt;
            page = page_next;
        }
        // No copy may still be in flight when the CTA ends, whatever the
        // other warps did.
        const WaitCtx dc{p.status, nullptr};
        for (int t = max(0, gt - S); t < gt; ++t) fa_wait(&bar_k[t % S], (t / S) & 1, 102, dc);
        for (int t = max(0, vt - S); t < vt; ++t) fa_wait(&bar_v[t % S], (t / S) & 1, 103, dc);
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------- MMAs
        if (lane == 0) {
            constexpr uint32_t idesc_s =
                F8 ? idesc_e4m3_f32(128, N) : idesc_bf16_f32(128, N, false, false);
            constexpr uint32_t idesc_o =
                F8 ? idesc_e4m3_f32(128, N, true) : idesc_bf16_f32(128, N, true, false);
            constexpr uint32_t kGroup = 8 * C::kSw;                  // 8 rows of a chunk
            const uint32_t skv = smem_u32(sKV), sq = smem_u32(sQ), sp = smem_u32(sP);
            auto desc = [&](uint32_t a, uint32_t lbo) {
                return C::kSw == 128 ? sdesc_sw128(a, lbo, kGroup) : sdesc_sw64(a, lbo, kGroup);
            };
            // O^T (+)= V_u^T P_u^T
            auto pv = [&](int u, bool first) -> bool {
                const int s = u % S;
                if (!fa_wait(&bar_p[u & 1], (u >> 1) & 1, 104, wc) ||
                    !fa_wait(&bar_v[s], (u / S) & 1, 105, wc))
                    return false;
                tc_fence_after();
                // V transposed: 32 (e4m3) or 16 keys a step; the next chunk of
                // columns (d = 64: K) is the leading-dimension stride
                const uint64_t vd =
                    desc(skv + s * 2 * TB, C::kChunks == 2 ? kTile * C::kSw : TB);
                const uint64_t pd = sdesc_sw128(sp + (u & 1) * C::kPBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < (F8 ? 4 : 8); ++kk) {
                    const uint64_t a = vd + (uint64_t)(kk * (F8 ? 32 : 16) * C::kSw >> 4);
                    const uint64_t b = pd + kmajor_step(kk, N * 128);
                    if (F8) mma_ss_f8(tmem + kColO, a, b, idesc_o, !first || kk > 0);
                    else mma_ss(tmem + kColO, a, b, idesc_o, !first || kk > 0);
                }
                mma_commit(&bar_pv[u & 1]);
                mma_commit(&bar_v_empty[s]);
                return true;
            };
            bool ok = true, first = false;        // first: tile gt - 1 begins its pair
            int gt = 0;
            for (int n = 0; ok && cur.left > 0; ++n) {
                const int tiles = cur.run();
                if (!fa_wait(&bar_q[n & 1], (n >> 1) & 1, 106, wc)) { ok = false; break; }
                tc_fence_after();
                const uint64_t qd = desc(sq + (n & 1) * C::kQBytes, 16);
                for (int t = 0; t < tiles; ++t, ++gt) {
                    const int s = gt % S;
                    if (!fa_wait(&bar_k[s], (gt / S) & 1, 107, wc)) { ok = false; break; }
                    tc_fence_after();
                    // S_t's buffer was read before P_{t-2} was complete
                    const uint64_t kd = desc(skv + s * 2 * TB + TB, 16);
#pragma unroll
                    for (int kk = 0; kk < C::kRowBytes / 32; ++kk) {
                        const uint64_t a = kd + kmajor_step(kk, kTile * 128);
                        const uint64_t b = qd + kmajor_step(kk, N * 128);
                        if (F8) mma_ss_f8(tmem + (gt & 1) * N, a, b, idesc_s, kk > 0);
                        else mma_ss(tmem + (gt & 1) * N, a, b, idesc_s, kk > 0);
                    }
                    mma_commit(&bar_s[gt & 1]);
                    mma_commit(&bar_k_empty[s]);
                    if (t + 1 == tiles) mma_commit(&bar_q_free[n & 1]);
                    // P V one tile behind, across pairs: the softmax warps have
                    // read a pair's O before they give the next pair's first P
                    if (gt > 0 && !pv(gt - 1, first)) { ok = false; break; }
                    first = t == 0;
                }
                cur.skip(p, tiles);
            }
            if (ok && gt > 0) ok = pv(gt - 1, first);
            if (!ok) {   // no MMA of this thread may still write TMEM at teardown
                mma_commit(&bar_drain);
                fa_wait(&bar_drain, 0, 108, WaitCtx{p.status, nullptr});
            }
        }
        __syncwarp();
    } else if (warp == 6) {
        // ---------------------------------------------------- query rows
        bool ok = true;
        for (int n = 0; ok && cur.left > 0; ++n) {
            if (n >= 2) ok = fa_wait_warp(&bar_q_free[n & 1], ((n >> 1) - 1) & 1, 109, wc);
            if (!ok) break;
            uint8_t* dst = sQ + (n & 1) * C::kQBytes;
            const __nv_bfloat16* src = p.q + ((long long)cur.b * p.Hkv + cur.g) * p.R * D;
            if constexpr (F8) {
                constexpr int E = D / 32;         // entries of a row per lane
                for (int r = 0; r < p.R; ++r) {
                    float x[E];
                    float amax = 0.0f;
                    const uint32_t* w = reinterpret_cast<const uint32_t*>(src + r * D) + lane * (E / 2);
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        const uint32_t u = __ldg(w + e);
                        x[2 * e] = __uint_as_float(u << 16);
                        x[2 * e + 1] = __uint_as_float(u & 0xffff0000u);
                    }
#pragma unroll
                    for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
                    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
                    // 2^k amax in [2^7, 2^8); k <= 120 (smaller rows keep fewer bits)
                    const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
                    const int k = min(7 - ex, 120);
                    const float up = __uint_as_float((uint32_t)(127 + k) << 23);
                    uint32_t c1 = 0, c2 = 0;
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float y0 = x[e] * up, y1 = x[e + 1] * up;
                        const uint32_t h = pack_e4m3x2(y0, y1);
                        float v[4];
                        unpack_e4m3x4(h, v);
                        c1 |= h << (8 * e);
                        c2 |= pack_e4m3x2(y0 - v[0], y1 - v[1]) << (8 * e);
                    }
                    const int byte = lane * E, unit = byte >> 4;
                    const int sw = C::kSw == 128 ? (r & 7) : ((r >> 1) & 3);
                    uint8_t* to = dst + r * C::kSw + ((unit ^ sw) << 4) + (byte & 15);
                    if (E == 4) {
                        *reinterpret_cast<uint32_t*>(to) = c1;
                        *reinterpret_cast<uint32_t*>(to + RP * C::kSw) = c2;
                    } else {
                        *reinterpret_cast<uint16_t*>(to) = (uint16_t)c1;
                        *reinterpret_cast<uint16_t*>(to + RP * C::kSw) = (uint16_t)c2;
                    }
                    // an infinite entry would saturate: the whole row becomes NaN
                    if (lane == 0)
                        q_scale[n & 1][r] =
                            ex == 128 ? CUDART_NAN_F
                                      : p.scale_log2 * __uint_as_float((uint32_t)(127 - k) << 23);
                }
                for (int r = p.R + lane; r < RP; r += 32) q_scale[n & 1][r] = 0.0f;
            } else {
                constexpr int U = D / 8;          // 16-byte units of a row
                for (int e = lane; e < p.R * U; e += 32) {
                    const int r = e / U, u = e % U;
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + e);
                    *reinterpret_cast<uint4*>(dst + (u >> 3) * (N * 128) + r * 128 +
                                              (((u & 7) ^ (r & 7)) << 4)) = w;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar_q[n & 1]);
            cur.skip(p, cur.run());
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax
        // Thread j holds key j of the tile.  A wait that gives up clears `ok`
        // and skips the later waits, but every thread stays in step with the
        // named barriers.
        const int j = threadIdx.x;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const int seg_shift = min(p.ps_shift, 7);
        // key j's scales in a stage: segment (j >> seg_shift), K's then V's
        const int ks_at = ((j >> seg_shift) << (seg_shift + 1)) + (j & ((1 << seg_shift) - 1));
        const int vs_at = ks_at + (1 << seg_shift);
        bool ok = true;
        int gt = 0;
        for (int n = 0; cur.left > 0; ++n) {
            const int tiles = cur.run();
            float m[RP], l[RP], qc[RP];
            if constexpr (F8) {
                ok = ok && fa_wait_warp(&bar_q[n & 1], (n >> 1) & 1, 110, wc);
#pragma unroll
                for (int r = 0; r < RP; ++r) qc[r] = q_scale[n & 1][r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar_q_free[n & 1]);
            }
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                m[r] = -CUDART_INF_F;
                l[r] = 0.0f;
            }
            for (int t = 0; t < tiles; ++t) {
                const int g_t = gt + t, s = g_t % S;
                const int key = (cur.t + t) * kTile + j;
                const int tile_end = (cur.t + t + 1) * kTile;
                const bool tail = tile_end > cur.len;
                uint32_t sr[N];
                ok = ok && fa_wait_warp(&bar_s[g_t & 1], (g_t >> 1) & 1, 111, wc);
                tc_fence_after();
                tmem_ld_cols<N>(tmem + lane_base + (g_t & 1) * N, sr);
                if (F8 || tail) ok = ok && fa_wait_warp(&bar_v[s], (g_t / S) & 1, 112, wc);
                float ks = 1.0f, vs = 1.0f, lv = 0.0f;
                if constexpr (F8) {
                    ks = sScale[s * 2 * kTile + ks_at];
                    vs = sScale[s * 2 * kTile + vs_at];
                    if (key >= cur.len) vs = 1.0f;          // may hold anything
                    lv = fmaxf(__log2f(fabsf(vs)), kMinLogScale);
                }
                float x[RP];
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    if constexpr (F8)
                        x[r] = (__uint_as_float(sr[r]) + __uint_as_float(sr[RP + r])) * (qc[r] * ks);
                    else
                        x[r] = __uint_as_float(sr[r]) * p.scale_log2;
                }
                if (tile_end > cur.len - (p.causal ? p.Nq - 1 : 0)) {
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const int end = p.causal ? cur.len - p.Nq + 1 + row_query[r] : cur.len;
                        if (key >= end) x[r] = -CUDART_INF_F;
                    }
                }
                // Does any score pass the running maximum by 2^kSlack?
                bool need = false;
#pragma unroll
                for (int r = 0; r < RP; ++r) need |= x[r] > m[r] + (C::kSlack - lv);
                if (named_bar_or(kSoftBar, 128, need)) {
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const int y = __reduce_max_sync(0xffffffffu, ordered(x[r] + lv));
                        if (lane == r) row_part[warp * RP + r] = from_ordered(y);
                    }
                    named_bar_sync(kSoftBar, 128);
                    float alpha[RP];
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float mx = fmaxf(fmax3(row_part[r], row_part[RP + r],
                                                     row_part[2 * RP + r]),
                                               fmaxf(row_part[3 * RP + r], m[r]));
                        alpha[r] = mx == m[r] ? 1.0f : ex2(m[r] - mx);
                        m[r] = mx;
                        l[r] *= alpha[r];
                    }
                    if (t > 0) {
                        ok = ok && fa_wait_warp(&bar_pv[(g_t - 1) & 1], ((g_t - 1) >> 1) & 1, 113,
                                                wc);
                        tc_fence_after();
                        if (warp * 32 < D) {
                            uint32_t ov[N];
                            tmem_ld_cols<N>(tmem + lane_base + kColO, ov);
#pragma unroll
                            for (int c = 0; c < N; ++c)
                                if (c < RP || F8)
                                    ov[c] = __float_as_uint(__uint_as_float(ov[c]) *
                                                            alpha[c % RP]);
#pragma unroll
                            for (int c = 0; c < N; c += 16) {
                                uint32_t part[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) part[e] = ov[c + e];
                                tmem_st16(tmem + lane_base + kColO + c, part);
                            }
                            tmem_st_wait();
                        }
                    }
                }
                // P's buffer: P_{t-2} V_{t-2} has read it
                if (g_t >= 2)
                    ok = ok && fa_wait_warp(&bar_pv[g_t & 1], ((g_t >> 1) - 1) & 1, 114, wc);
                uint8_t* pb = sP + (g_t & 1) * C::kPBytes;
                if constexpr (F8) {
                    uint8_t* to = pb + (j & 15);
                    const int unit = j >> 4;
                    const float wv = vs * C::kPScale;
#pragma unroll
                    for (int r = 0; r < RP; r += 2) {
                        float w[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float mu = m[r + h] == -CUDART_INF_F ? 0.0f : m[r + h];
                            const float e = ex2(x[r + h] - mu);
                            l[r + h] += e;
                            w[h] = e * wv;
                        }
                        const uint32_t h1 = pack_e4m3x2(w[0], w[1]);
                        float v[4];
                        unpack_e4m3x4(h1, v);
                        const uint32_t h2 = pack_e4m3x2(w[0] - v[0], w[1] - v[1]);
                        uint8_t* a0 = to + r * 128 + ((unit ^ (r & 7)) << 4);
                        uint8_t* a1 = to + (r + 1) * 128 + ((unit ^ ((r + 1) & 7)) << 4);
                        a0[0] = (uint8_t)h1;
                        a1[0] = (uint8_t)(h1 >> 8);
                        a0[RP * 128] = (uint8_t)h2;
                        a1[RP * 128] = (uint8_t)(h2 >> 8);
                    }
                } else {
                    uint8_t* to = pb + (j >> 6) * (N * 128) + (j & 7) * 2;
                    const int unit = (j & 63) >> 3;
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float mu = m[r] == -CUDART_INF_F ? 0.0f : m[r];
                        const float e = ex2(x[r] - mu);
                        l[r] += e;
                        *reinterpret_cast<__nv_bfloat16*>(to + r * 128 + ((unit ^ (r & 7)) << 4)) =
                            __float2bfloat16_rn(e);
                    }
                }
                if (tail && key >= cur.len) {
                    // V rows past the sequence may hold NaN, which a weight of
                    // zero does not silence
                    uint8_t* vrow = sKV + s * 2 * TB + j * C::kSw;
#pragma unroll
                    for (int c = 0; c < C::kChunks; ++c)
#pragma unroll
                        for (int u = 0; u < C::kSw / 16; ++u)
                            *reinterpret_cast<uint4*>(vrow + c * (kTile * C::kSw) + u * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(&bar_p[g_t & 1]);
            }
            // The pair's part: O / l, and LSE (or O and LSE themselves).
            const int g_last = gt + tiles - 1;
            ok = ok && fa_wait_warp(&bar_pv[g_last & 1], (g_last >> 1) & 1, 115, wc);
            tc_fence_after();
            uint32_t ov[N];
            tmem_ld_cols<N>(tmem + lane_base + kColO, ov);
            int row;
            const float total = warp_row_sums<RP>(l, lane, row);
            row_part[warp * RP + row] = total;            // several lanes, one value
            named_bar_sync(kSoftBar, 128);
            const int pair = cur.b * p.Hkv + cur.g;
            const bool whole = tiles == tiles_of(cur.len);
            const long long slot = (long long)blockIdx.x + pair;
            const long long out_row = whole ? (long long)pair * p.R : slot * p.R;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                if (r >= p.R) break;
                const float lr = (row_part[r] + row_part[RP + r]) +
                                 (row_part[2 * RP + r] + row_part[3 * RP + r]);
                const float y = F8 ? __uint_as_float(ov[r]) + __uint_as_float(ov[(RP + r) % N])
                                   : __uint_as_float(ov[r]);
                const float out = lr == 0.0f ? 0.0f : y / (lr * C::kPScale);
                if (warp * 32 < D) {
                    if (whole)
                        p.o[(out_row + r) * D + j] = __float2bfloat16_rn(out);
                    else
                        p.part_o[(out_row + r) * D + j] = out;
                }
                if (j == r) {
                    const float lse2 = lr == 0.0f ? -CUDART_INF_F : m[r] + log2f(lr);
                    if (whole)
                        p.lse[out_row + r] = lse2 * kLn2;
                    else
                        p.part_lse[out_row + r] = lse2;
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
}

// One warp per query row of the pairs that several CTAs share: the parts
// weighted by exp(LSE_s - LSE), in slot order.  Rows of empty sequences are
// written here.  Where a row's parts lie follows from the lengths alone and is
// found while the split kernel still runs; after it, the parts' LSEs and the
// first kPre parts of O come in one round trip.
template <int D>
__global__ void __launch_bounds__(256) fa_paged_combine_kernel(const PagedParams p, int rows) {
    constexpr int E = D / 32, kPre = 8;
    const int row = (int)((blockIdx.x * 256 + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    const int pair = min(row, rows - 1) / p.R, r = row - pair * p.R;
    const int b = pair / p.Hkv, g = pair - b * p.Hkv;
    int b0, b1, at, upto;
    const int T = list_length(p, lane, b0, b1, at, upto);
    const int tiles = tiles_of(clamped_len(p, b));
    for (int x = b0; x < b1 && x < b; ++x) at += tiles_of(clamped_len(p, x)) * p.Hkv;
    // the lane whose sequences b is one of
    const int first = __shfl_sync(0xffffffffu, at, b / ((p.B + 31) / 32)) + g * tiles;
    const int nc = min(p.ctas, T);
    const int c0 = tiles ? cta_of_tile(first, T, nc) : 0;
    const int parts = tiles ? cta_of_tile(first + tiles - 1, T, nc) - c0 + 1 : 0;
    // Every thread waits here, also those with nothing to join: this grid must
    // not end before the split kernel, whose results the next one in the
    // stream may read.
    pdl_wait();
    if (row >= rows || parts == 1) return;
    __nv_bfloat16* o = p.o + (long long)row * D + lane;
    if (parts == 0) {
#pragma unroll
        for (int c = 0; c < E; ++c) o[32 * c] = __float2bfloat16_rn(0.0f);
        if (lane == 0) p.lse[row] = -CUDART_INF_F;
        return;
    }
    const long long slot = (long long)c0 + pair;
    const float* lp = p.part_lse + slot * p.R + r;
    const float* op = p.part_o + (slot * p.R + r) * D + lane;
    const long long lstep = p.R, ostep = (long long)p.R * D;
    const float l0 = lane < parts ? __ldcg(lp + lane * lstep) : -CUDART_INF_F;
    float pre[kPre][E];
#pragma unroll
    for (int k = 0; k < kPre; ++k)
#pragma unroll
        for (int c = 0; c < E; ++c) pre[k][c] = k < parts ? __ldcg(op + k * ostep + 32 * c) : 0.0f;
    float mx = l0;
    for (int s = lane + 32; s < parts; s += 32) mx = fmaxf(mx, __ldcg(lp + s * lstep));
    mx = from_ordered(__reduce_max_sync(0xffffffffu, ordered(mx)));
    if (mx == -CUDART_INF_F) mx = 0.0f;
    float acc[E], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < E; ++c) acc[c] = 0.0f;
    for (int base = 0; base < parts; base += 32) {
        const int s = base + lane;
        const float ls = base == 0 ? l0 : (s < parts ? __ldcg(lp + s * lstep) : -CUDART_INF_F);
        const float w = ex2(ls - mx);
        const int cnt = min(32, parts - base);
        sum += w;
        int k = 0;
        if (base == 0) {
#pragma unroll
            for (; k < kPre; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
                for (int c = 0; c < E; ++c) acc[c] = fmaf(wk, pre[k][c], acc[c]);
            }
        }
#pragma unroll 8
        for (; k < cnt; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
#pragma unroll
            for (int c = 0; c < E; ++c)
                acc[c] = fmaf(wk, __ldcg(op + (base + k) * ostep + 32 * c), acc[c]);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
    for (int c = 0; c < E; ++c)
        o[32 * c] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc[c] / sum);
    if (lane == 0) p.lse[row] = sum == 0.0f ? -CUDART_INF_F : (mx + log2f(sum)) * kLn2;
}

template <int D, bool F8, int RP>
cudaError_t launch_split(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                         cudaStream_t stream) {
    using C = Cfg<D, F8, RP>;
    static_assert(C::kSmem + 2048 <= 227 * 1024, "shared memory of one CTA");
    auto kern = fa_decode_paged_kernel<D, F8, RP>;
    static std::atomic<unsigned long long> configured{0};     // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!((configured.load(std::memory_order_acquire) >> dev) & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        configured.fetch_or(1ull << dev, std::memory_order_release);
    }
    // no more CTAs than there can be tiles
    const long long most = (long long)p.B * p.Hkv * (((p.max_pages << p.ps_shift) + kTile - 1) / kTile);
    long long grid = (long long)(device_sm_count() > 0 ? device_sm_count() : 152) * C::kCtas;
    if (grid > kPagedMaxCtas) grid = kPagedMaxCtas;
    if (grid > most) grid = most;
    p.ctas = (int)grid;
    count_launch();
    kern<<<(unsigned)grid, kThreads, C::kSmem, stream>>>(tk, tv, p);
    return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, PagedParams& p,
                        cudaStream_t stream) {
    if (p.R <= 8) return launch_split<D, F8, 8>(tk, tv, p, stream);
    if (p.R <= 16) return launch_split<D, F8, 16>(tk, tv, p, stream);
    return launch_split<D, F8, 32>(tk, tv, p, stream);
}

template <int D>
cudaError_t launch_combine(const PagedParams& p, cudaStream_t stream) {
    const int rows = p.B * p.Hkv * p.R;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    // its blocks come in while the split kernel still runs and wait for it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fa_paged_combine_kernel<D>, p, rows);
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
    cudaError_t e;
    if (c.d == 128)
        e = f8 ? launch_rows<128, true>(tk, tv, p, stream) : launch_rows<128, false>(tk, tv, p, stream);
    else
        e = f8 ? launch_rows<64, true>(tk, tv, p, stream) : launch_rows<64, false>(tk, tv, p, stream);
    if (e != cudaSuccess) return e;
    return c.d == 128 ? launch_combine<128>(p, stream) : launch_combine<64>(p, stream);
}

}  // namespace fa
