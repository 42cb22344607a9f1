// Paged key/value cache: writing new rows into the pages (bf16 as they are, or
// quantised to e4m3 with one scale per token and head) and reading cached rows
// back as contiguous bf16.
//
// Position x of sequence b lives in page block_table[b][x / page_size], row
// x % page_size; a page holds [Hkv][page_size][d].  The quantiser, over the d
// values of one K or V row: amax = max |x|, scale = amax / 448, code =
// e4m3(x * (448 / amax)), both quotients in fp32 (scale 0 and codes 0 for a
// row of zeros; a nonzero amax below 2^-100 counts as 2^-100, so that the
// quotient stays finite).  448 is e4m3's largest value, so the row's largest
// magnitude lands on it and every other one rounds by at most 2^-4 of itself.
//
// Both directions are copies bound by HBM, as long as the instructions around
// them stay few.  A warp takes up to 32 rows of K and V.  Each lane finds one
// row's place once (its sequence, its page); then D / 8 lanes share a row, 16
// bytes of bf16 each, and get the place by shuffles, the rows of kBatch passes in
// flight together.  The maxima of K and of V travel as one bf16 pair, and one
// division gives all four quotients of a row: a quarter of its lanes each takes
// 448 / amax or amax / 448 of K or of V.  The scales are kept until the warp's
// rows are done and leave as whole runs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;
// Up to here a warp takes one pass of rows (the short form): they spread over more
// SMs, and none waits for a second batch.  Both forms, short and long, us in a graph of
// calls on inputs larger than L2 (rows of K, and of V; pages of 16):
//                          8192         16384        32768        49152        65536
//   e4m3 append   d = 128  4.55  6.43   5.49  6.85   7.85  8.26   10.3  10.0   12.5  11.7
//                 d = 64   3.02  4.74   4.54  6.34   5.44  6.76   6.95  7.81   7.92  8.18
//   bf16 append   d = 128  4.30  4.33   5.78  5.85   8.05  8.00   10.8  10.6   13.1  13.1
//                 d = 64   3.64  3.90   4.62  4.71   5.70  5.82   7.20  7.07   8.08  7.97
//   bf16 gather   d = 128  4.62  4.75   5.78  5.83   8.19  8.07   10.9  10.5   13.5  13.2
//                 d = 64   3.55  3.80   4.62  4.77   5.67  5.85   7.27  7.13   8.20  7.99
//   e4m3 gather   d = 128  4.37  4.47   5.31  5.27   7.47  6.97   9.79  8.56   12.0  10.3
//                 d = 64   2.95  3.30   4.33  4.54   5.25  5.30   6.65  6.24   7.56  7.08
template <bool F8, bool APPEND>
constexpr unsigned kFewRows = F8 && APPEND ? 49152 : 16384;

// n / d for 31-bit n: q = floor(n * floor(2^32 / d) / 2^32) is the quotient or
// one less.
struct Divider {
    unsigned d, inv;
    explicit Divider(unsigned d_) : d(d_), inv(d_ == 1 ? 0u : (unsigned)((1ull << 32) / d_)) {}
    __device__ __forceinline__ unsigned operator()(unsigned n) const {
        if (d == 1) return n;
        const unsigned q = __umulhi(n, inv);
        return q + (n - q * d >= d);
    }
};

struct MoveParams {
    void* k;                  // contiguous side: [B][Hkv][N][d], or packed [Hkv][total][d]
    void* v;
    void* k_pages;
    void* v_pages;
    float* scales;            // e4m3: [n_pages][Hkv][2][page_size]
    const int* table;
    const int* starts;
    const int* counts;        // dense: rows of each sequence; packed: cu_seqlens [B + 1]
    int B, Hkv, N, total, packed, n_pages, ps_shift, max_pages;
    Divider by_run, by_heads; // rows of a head in a row (N or total); Hkv
    unsigned rows;            // rows of the contiguous side
};

// Row r of the contiguous side in the pool: page * Hkv + g in `head` and the row
// of the page, or false when there is none: padding, or a position or page
// outside the table or the pool.
__device__ __forceinline__ bool find_place(const MoveParams& p, unsigned r, int& head, int& row) {
    if (r >= p.rows) return false;
    const unsigned run = p.by_run(r);
    const int at = (int)(r - run * p.by_run.d);
    int b, g, i;
    if (p.packed) {
        // the last sequence that begins at or before row `at`
        g = (int)run;
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__ldg(p.counts + mid) <= at) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        const int first = __ldg(p.counts + b);
        i = at - first;
        if (first < 0 || i < 0 || i >= p.N || at >= __ldg(p.counts + b + 1)) return false;
    } else {
        b = (int)p.by_heads(run);
        g = (int)run - b * p.Hkv;
        i = at;
        if (i >= __ldg(p.counts + b)) return false;
    }
    const long long pos = (long long)__ldg(p.starts + b) + i;
    if (pos < 0 || (pos >> p.ps_shift) >= p.max_pages) return false;
    const int page = __ldg(p.table + (long long)b * p.max_pages + (pos >> p.ps_shift));
    if ((unsigned)page >= (unsigned)p.n_pages) return false;
    head = page * p.Hkv + g;
    row = (int)(pos & ((1 << p.ps_shift) - 1));
    return true;
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // ignores NaN
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_abs8(const uint4& w) {
    const uint32_t m = 0x7fff7fffu;
    return max_bf16x2(max_bf16x2(w.x & m, w.y & m), max_bf16x2(w.z & m, w.w & m));
}

__device__ __forceinline__ uint2 encode8(const uint4& w, float inv) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16) * inv;
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u) * inv;
    }
    return make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
}

// Eight e4m3 codes times the row's scale, as eight bf16 values.
__device__ __forceinline__ uint4 decode8(const uint2& c, float scale) {
    float x[4], y[4];
    unpack_e4m3x4(c.x, x);
    unpack_e4m3x4(c.y, y);
    return make_uint4(
        pack_bf16x2(x[0] * scale, x[1] * scale), pack_bf16x2(x[2] * scale, x[3] * scale),
        pack_bf16x2(y[0] * scale, y[1] * scale), pack_bf16x2(y[2] * scale, y[3] * scale));
}

// Passes whose loads are in flight together, and rounds of them: a warp moves
// kRounds * kBatch * 256 / D rows of K and of V (the long form: 8 rows of d = 128 and 16
// of d = 64, twice as many where it quantises).
template <int D, bool F8, bool APPEND, int kBatch, int kRounds>
__global__ void __launch_bounds__(kThreads)
fa_kv_move_kernel(const __grid_constant__ MoveParams p) {
    constexpr int LPR = D / 8, RPP = 32 / LPR;       // lanes a row, rows a pass
    constexpr int kWarpRows = kRounds * kBatch * RPP;
    static_assert(kWarpRows <= 32, "a lane finds one row's place");
    const int lane = threadIdx.x & 31, part = lane % LPR, sub = lane / LPR;
    const unsigned r0 = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (unsigned)kWarpRows;
    int my_head = -1, my_row = 0;
    if (lane >= kWarpRows || !find_place(p, r0 + lane, my_head, my_row)) my_head = -1;
    if (!__any_sync(0xffffffffu, my_head >= 0)) return;
    const long long my_scale = ((long long)my_head << (p.ps_shift + 1)) + my_row;
    float ks = 0.0f, vs = 0.0f;                      // e4m3: scales of this lane's own row
    if (F8 && !APPEND && my_head >= 0) {
        ks = __ldg(p.scales + my_scale);
        vs = __ldg(p.scales + my_scale + (1LL << p.ps_shift));
    }
#pragma unroll 1
    for (int round = 0; round < kRounds; ++round) {
        long long flat[kBatch], paged[kBatch];       // in units of this lane's 8 values
        bool ok[kBatch];
        uint4 kw[kBatch], vw[kBatch];
        uint2 kc[kBatch], vc[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int src = (round * kBatch + i) * RPP + sub;
            const int head = __shfl_sync(0xffffffffu, my_head, src);
            const int row = __shfl_sync(0xffffffffu, my_row, src);
            ok[i] = head >= 0;
            flat[i] = (long long)(r0 + src) * LPR + part;
            paged[i] = (((long long)head << p.ps_shift) + row) * LPR + part;
            kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
            kc[i] = vc[i] = make_uint2(0u, 0u);
            if (!ok[i]) continue;
            if (APPEND) {
                kw[i] = __ldg(static_cast<const uint4*>(p.k) + flat[i]);
                vw[i] = __ldg(static_cast<const uint4*>(p.v) + flat[i]);
            } else if (F8) {
                kc[i] = __ldg(static_cast<const uint2*>(p.k_pages) + paged[i]);
                vc[i] = __ldg(static_cast<const uint2*>(p.v_pages) + paged[i]);
            } else {
                kw[i] = __ldg(static_cast<const uint4*>(p.k_pages) + paged[i]);
                vw[i] = __ldg(static_cast<const uint4*>(p.v_pages) + paged[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int pass = round * kBatch + i;
            if constexpr (F8 && APPEND) {
                // (K, V) maxima over the row's lanes
                const uint32_t a = max_abs8(kw[i]), b = max_abs8(vw[i]);
                uint32_t m = max_bf16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1)
                    m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, off));
                // quarter 0: 448 / amax of K, 1: amax / 448 of K; 2, 3: of V
                const int quarter = part / (LPR / 4);
                float amax = __uint_as_float(quarter < 2 ? m << 16 : m & 0xffff0000u);
                const bool zero = amax == 0.0f;
                amax = fmaxf(amax, 0x1p-100f);
                float quot = (quarter & 1 ? amax : 448.0f) / (quarter & 1 ? 448.0f : amax);
                if (zero) quot = 0.0f;
                const int base = lane - part;
                const float kinv = __shfl_sync(0xffffffffu, quot, base);
                const float vinv = __shfl_sync(0xffffffffu, quot, base + LPR / 2);
                // this pass's scales to the lanes whose rows they are
                const int from = (lane % RPP) * LPR;
                const float ksc = __shfl_sync(0xffffffffu, quot, from + LPR / 4);
                const float vsc = __shfl_sync(0xffffffffu, quot, from + LPR / 4 * 3);
                if (lane / RPP == pass) {
                    ks = ksc;
                    vs = vsc;
                }
                if (ok[i]) {
                    static_cast<uint2*>(p.k_pages)[paged[i]] = encode8(kw[i], kinv);
                    static_cast<uint2*>(p.v_pages)[paged[i]] = encode8(vw[i], vinv);
                }
            } else if constexpr (APPEND) {
                if (ok[i]) {
                    static_cast<uint4*>(p.k_pages)[paged[i]] = kw[i];
                    static_cast<uint4*>(p.v_pages)[paged[i]] = vw[i];
                }
            } else {
                if constexpr (F8) {
                    const float ksc = __shfl_sync(0xffffffffu, ks, pass * RPP + sub);
                    const float vsc = __shfl_sync(0xffffffffu, vs, pass * RPP + sub);
                    kw[i] = decode8(kc[i], ksc);
                    vw[i] = decode8(vc[i], vsc);
                }
                if (ok[i]) {
                    static_cast<uint4*>(p.k)[flat[i]] = kw[i];
                    static_cast<uint4*>(p.v)[flat[i]] = vw[i];
                }
            }
        }
    }
    if (F8 && APPEND && my_head >= 0) {
        p.scales[my_scale] = ks;
        p.scales[my_scale + (1LL << p.ps_shift)] = vs;
    }
}

template <int D, bool F8, bool APPEND, int kBatch, int kRounds>
cudaError_t launch(const MoveParams& p, cudaStream_t stream) {
    constexpr unsigned per_block = kThreads / 32 * kRounds * kBatch * (256 / D);
    count_launch();
    fa_kv_move_kernel<D, F8, APPEND, kBatch, kRounds>
        <<<(p.rows + per_block - 1) / per_block, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// The long form: four passes in flight; the quantiser's work is long enough for a
// second round on the same places (16 packed prompts of 128 to 4096 tokens, H16
// d128: 76.6 us with two rounds, 84.8 with one, 78.6 with four), copies are not
// (32K tokens of 8 heads read back from e4m3: 122.7 us with one round, 124.5 with
// four).
template <int D, bool F8, bool APPEND>
cudaError_t launch_rows(const MoveParams& p, cudaStream_t stream) {
    if (p.rows <= kFewRows<F8, APPEND>) return launch<D, F8, APPEND, 1, 1>(p, stream);
    return launch<D, F8, APPEND, 4, F8 && APPEND ? 2 : 1>(p, stream);
}

template <int D>
cudaError_t launch_type(const MoveParams& p, bool append, cudaStream_t stream) {
    if (append)
        return p.scales ? launch_rows<D, true, true>(p, stream)
                        : launch_rows<D, false, true>(p, stream);
    return p.scales ? launch_rows<D, true, false>(p, stream)
                    : launch_rows<D, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_kv_move(const PagedCache& c, void* k, void* v, const int* starts,
                           const int* counts, int B, int N, int total, bool packed, bool append,
                           cudaStream_t stream) {
    const unsigned run = (unsigned)(packed ? total : N);
    MoveParams p{k,
                 v,
                 const_cast<void*>(c.k_pages),
                 const_cast<void*>(c.v_pages),
                 const_cast<float*>(c.scales),
                 c.table,
                 starts,
                 counts,
                 B,
                 c.Hkv,
                 N,
                 total,
                 packed,
                 c.n_pages,
                 c.ps_shift,
                 c.max_pages,
                 Divider(run),
                 Divider((unsigned)c.Hkv),
                 (unsigned)((packed ? 1LL : (long long)B) * c.Hkv * run)};
    if (c.d == 128) return launch_type<128>(p, append, stream);
    return launch_type<64>(p, append, stream);
}

}  // namespace fa
