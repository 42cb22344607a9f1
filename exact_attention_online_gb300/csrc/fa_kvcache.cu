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
// Both directions are copies bound by HBM: D / 8 lanes hold one row, 16 bytes
// of bf16 each, so that a warp's accesses are whole 128-byte lines on the
// contiguous side and on the page side (rows of a page are adjacent), and the
// row's maximum is D / 8 lanes of one shuffle reduction.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreads = 256;

struct MoveParams {
    void* k;                  // contiguous side: [B][Hkv][N][d], or packed [Hkv][total][d]
    void* v;
    void* k_pages;
    void* v_pages;
    float* scales;            // e4m3: [n_pages][Hkv][2][page_size]
    const int* table;
    const int* starts;
    const int* counts;        // dense: rows of each sequence; packed: cu_seqlens [B + 1]
    int Hkv, N, total, packed, n_pages, ps_shift, max_pages;
    unsigned rows;            // B * Hkv * N
};

// Where row (b, g, i) sits on both sides, or false when there is none: i past
// the sequence's count, or a position or page outside the table or the pool.
struct Place {
    long long flat;           // row index on the contiguous side
    long long paged;          // row index in the pool, (page * Hkv + g) * page_size + row
    long long scale;          // its K scale's index; V's is page_size further
};

__device__ __forceinline__ bool find_place(const MoveParams& p, unsigned r, Place& at) {
    if (r >= p.rows) return false;
    const unsigned bg = r / (unsigned)p.N;
    const int i = (int)(r - bg * (unsigned)p.N);
    const int b = (int)(bg / (unsigned)p.Hkv), g = (int)(bg - (unsigned)b * (unsigned)p.Hkv);
    if (p.packed) {
        int t0;
        const int n = packed_seq(p.counts, b, p.N, p.total, t0);
        if (i >= n) return false;
        at.flat = (long long)g * p.total + t0 + i;
    } else {
        if (i >= __ldg(p.counts + b)) return false;
        at.flat = r;
    }
    const long long pos = (long long)__ldg(p.starts + b) + i;
    if (pos < 0 || (pos >> p.ps_shift) >= p.max_pages) return false;
    const int page = __ldg(p.table + (long long)b * p.max_pages + (pos >> p.ps_shift));
    if ((unsigned)page >= (unsigned)p.n_pages) return false;
    const long long pg = (long long)page * p.Hkv + g;
    const int row = (int)(pos & ((1 << p.ps_shift) - 1));
    at.paged = (pg << p.ps_shift) + row;
    at.scale = (pg << (p.ps_shift + 1)) + row;
    return true;
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
}

// Eight values of a row spread over LPR lanes: the row's scale, and the codes.
template <int LPR>
__device__ __forceinline__ uint2 quantise8(const uint4& w, float& scale) {
    float x[8];
    bf16x8_to_f32(w, x);
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (amax > 0.0f) amax = fmaxf(amax, 0x1p-100f);
    scale = amax / 448.0f;
    const float inv = amax > 0.0f ? 448.0f / amax : 0.0f;
    return make_uint2(pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// Four e4m3 codes times the row's scale, as four bf16 values.
__device__ __forceinline__ uint2 dequantise4(uint32_t codes, float scale) {
    float x[4];
    unpack_e4m3x4(codes, x);
    return make_uint2(pack_bf16x2(x[0] * scale, x[1] * scale),
                      pack_bf16x2(x[2] * scale, x[3] * scale));
}

// U rows of K and of V per group of D / 8 lanes, all loads issued before the
// first use.
template <int D, bool F8, int U>
__global__ void __launch_bounds__(kThreads) fa_kv_append_kernel(const MoveParams p) {
    constexpr int LPR = D / 8, RPB = kThreads / LPR;
    const int lane = threadIdx.x % LPR;
    const unsigned r0 = blockIdx.x * (unsigned)(RPB * U) + threadIdx.x / LPR;
    Place at[U];
    bool ok[U];
    uint4 kw[U], vw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ok[u] = find_place(p, r0 + u * RPB, at[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (ok[u]) {
            kw[u] = __ldg(static_cast<const uint4*>(p.k) + at[u].flat * LPR + lane);
            vw[u] = __ldg(static_cast<const uint4*>(p.v) + at[u].flat * LPR + lane);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if constexpr (F8) {
            float ks, vs;
            const uint2 kc = quantise8<LPR>(kw[u], ks), vc = quantise8<LPR>(vw[u], vs);
            if (ok[u]) {
                static_cast<uint2*>(p.k_pages)[at[u].paged * LPR + lane] = kc;
                static_cast<uint2*>(p.v_pages)[at[u].paged * LPR + lane] = vc;
                if (lane == 0) p.scales[at[u].scale] = ks;
                if (lane == 1) p.scales[at[u].scale + (1LL << p.ps_shift)] = vs;
            }
        } else if (ok[u]) {
            static_cast<uint4*>(p.k_pages)[at[u].paged * LPR + lane] = kw[u];
            static_cast<uint4*>(p.v_pages)[at[u].paged * LPR + lane] = vw[u];
        }
    }
}

template <int D, bool F8, int U>
__global__ void __launch_bounds__(kThreads) fa_kv_gather_kernel(const MoveParams p) {
    constexpr int LPR = D / 8, RPB = kThreads / LPR;
    const int lane = threadIdx.x % LPR;
    const unsigned r0 = blockIdx.x * (unsigned)(RPB * U) + threadIdx.x / LPR;
    Place at[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) ok[u] = find_place(p, r0 + u * RPB, at[u]);
    if constexpr (F8) {
        uint2 kc[U], vc[U];
        float ks[U], vs[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok[u]) {
                kc[u] = __ldg(static_cast<const uint2*>(p.k_pages) + at[u].paged * LPR + lane);
                vc[u] = __ldg(static_cast<const uint2*>(p.v_pages) + at[u].paged * LPR + lane);
                ks[u] = __ldg(p.scales + at[u].scale);
                vs[u] = __ldg(p.scales + at[u].scale + (1LL << p.ps_shift));
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok[u]) {
                const uint2 k0 = dequantise4(kc[u].x, ks[u]), k1 = dequantise4(kc[u].y, ks[u]);
                const uint2 v0 = dequantise4(vc[u].x, vs[u]), v1 = dequantise4(vc[u].y, vs[u]);
                static_cast<uint4*>(p.k)[at[u].flat * LPR + lane] = make_uint4(k0.x, k0.y, k1.x, k1.y);
                static_cast<uint4*>(p.v)[at[u].flat * LPR + lane] = make_uint4(v0.x, v0.y, v1.x, v1.y);
            }
    } else {
        uint4 kw[U], vw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok[u]) {
                kw[u] = __ldg(static_cast<const uint4*>(p.k_pages) + at[u].paged * LPR + lane);
                vw[u] = __ldg(static_cast<const uint4*>(p.v_pages) + at[u].paged * LPR + lane);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok[u]) {
                static_cast<uint4*>(p.k)[at[u].flat * LPR + lane] = kw[u];
                static_cast<uint4*>(p.v)[at[u].flat * LPR + lane] = vw[u];
            }
    }
}

constexpr int kRowsInFlight = 4;

template <int D, bool F8>
cudaError_t launch_move(const MoveParams& p, bool append, cudaStream_t stream) {
    constexpr int U = kRowsInFlight;
    constexpr unsigned per_block = kThreads / (D / 8) * U;
    const unsigned blocks = (p.rows + per_block - 1) / per_block;
    count_launch();
    if (append)
        fa_kv_append_kernel<D, F8, U><<<blocks, kThreads, 0, stream>>>(p);
    else
        fa_kv_gather_kernel<D, F8, U><<<blocks, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_move(const PagedCache& c, void* k, void* v, const int* starts,
                           const int* counts, int B, int N, int total, bool packed, bool append,
                           cudaStream_t stream) {
    MoveParams p;
    p.k = k;
    p.v = v;
    p.k_pages = const_cast<void*>(c.k_pages);
    p.v_pages = const_cast<void*>(c.v_pages);
    p.scales = const_cast<float*>(c.scales);
    p.table = c.table;
    p.starts = starts;
    p.counts = counts;
    p.Hkv = c.Hkv;
    p.N = N;
    p.total = total;
    p.packed = packed;
    p.n_pages = c.n_pages;
    p.ps_shift = c.ps_shift;
    p.max_pages = c.max_pages;
    p.rows = (unsigned)((long long)B * c.Hkv * N);
    if (c.d == 128)
        return c.scales ? launch_move<128, true>(p, append, stream)
                        : launch_move<128, false>(p, append, stream);
    return c.scales ? launch_move<64, true>(p, append, stream)
                    : launch_move<64, false>(p, append, stream);
}

}  // namespace fa
