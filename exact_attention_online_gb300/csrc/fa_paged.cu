// Decoding attention over a paged key/value cache: Nq new query rows of each
// sequence against the rows its block table names, sequences of different
// lengths, pages in bf16 or in e4m3 with one scale per token and head.
//
// Simple form: one CTA per query row; its warps take the visible keys in
// turn, each with its own running maximum and sum, and are joined at the end
// by their log-sum-exp weights.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;

struct PagedParams {
    const __nv_bfloat16* q;
    const void* k_pages;
    const void* v_pages;
    const float* scales;
    const int* table;
    const int* seqlens;
    __nv_bfloat16* o;
    float* lse;
    int H, Hkv, Nq, n_pages, ps_shift, max_pages, causal;
    float scale_log2;
};

template <int D, bool F8>
__device__ __forceinline__ void load_row(const void* pages, long long row, int lane, float scale,
                                         float (&x)[D / 32]) {
    constexpr int E = D / 32;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const long long at = row * D + lane * E + e;
        if constexpr (F8) {
            float y[4];
            unpack_e4m3x4(static_cast<const uint8_t*>(pages)[at], y);
            x[e] = y[0] * scale;
        } else {
            x[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(pages)[at]);
        }
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kWarps * 32) fa_decode_paged_kernel(const PagedParams p) {
    constexpr int E = D / 32;
    const long long row = blockIdx.x;                 // (b * H + h) * Nq + i
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int i = (int)(row % p.Nq);
    const int h = (int)(row / p.Nq % p.H), b = (int)(row / p.Nq / p.H);
    const int g = h / (p.H / p.Hkv);
    const int cap = p.max_pages << p.ps_shift;
    const int len = min(max(__ldg(p.seqlens + b), 0), cap);
    const int end = p.causal ? max(0, len - p.Nq + i + 1) : len;   // keys 0 .. end - 1
    float q[E], acc[E];
    float m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * D + lane * E + e]) * p.scale_log2;
        acc[e] = 0.0f;
    }
    for (int j = warp; j < end; j += kWarps) {
        const int page = __ldg(p.table + (long long)b * p.max_pages + (j >> p.ps_shift));
        if ((unsigned)page >= (unsigned)p.n_pages) continue;
        const long long pg = (long long)page * p.Hkv + g;
        const int pr = j & ((1 << p.ps_shift) - 1);
        float ks = 1.0f, vs = 1.0f, x[E];
        if constexpr (F8) {
            ks = __ldg(p.scales + (pg << (p.ps_shift + 1)) + pr);
            vs = __ldg(p.scales + (pg << (p.ps_shift + 1)) + (1 << p.ps_shift) + pr);
        }
        load_row<D, F8>(p.k_pages, (pg << p.ps_shift) + pr, lane, ks, x);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        const float mn = fmaxf(m, s);
        const float a = (m == -CUDART_INF_F) ? 0.0f : exp2f(m - mn);
        const float w = (s == -CUDART_INF_F) ? 0.0f : exp2f(s - mn);   // a NaN stays one
        load_row<D, F8>(p.v_pages, (pg << p.ps_shift) + pr, lane, vs, x);
        m = mn;
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e] * a);
    }
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    float mx = -CUDART_INF_F, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
    for (int w = 0; w < kWarps; ++w) sum += sl[w] != 0.0f ? sl[w] * exp2f(sm[w] - mx) : 0.0f;
    for (int c = threadIdx.x; c < D; c += kWarps * 32) {
        float y = 0.0f;
        for (int w = 0; w < kWarps; ++w) y += sl[w] != 0.0f ? so[w][c] * exp2f(sm[w] - mx) : 0.0f;
        p.o[row * D + c] = __float2bfloat16_rn(sum != 0.0f ? y / sum : 0.0f);
    }
    if (threadIdx.x == 0) p.lse[row] = sum != 0.0f ? (mx + log2f(sum)) * kLn2 : -CUDART_INF_F;
}

}  // namespace

size_t paged_workspace_bytes(int B, int Hkv, int R, int d) {
    const size_t slots = (size_t)kPagedMaxCtas + (size_t)B * Hkv;
    return (slots * R * d * 4 + 255) / 256 * 256 + (slots * R * 4 + 255) / 256 * 256 +
           (size_t)B * Hkv * 8;
}

cudaError_t launch_fwd_decode_paged(const PagedCache& c, const void* q, void* o, float* lse,
                                    const int* seqlens, void* workspace, int B, int H, int Nq,
                                    int causal, float scale, DeviceStatus* status,
                                    cudaStream_t stream) {
    PagedParams p;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_pages = c.k_pages;
    p.v_pages = c.v_pages;
    p.scales = c.scales;
    p.table = c.table;
    p.seqlens = seqlens;
    p.o = static_cast<__nv_bfloat16*>(o);
    p.lse = lse;
    p.H = H;
    p.Hkv = c.Hkv;
    p.Nq = Nq;
    p.n_pages = c.n_pages;
    p.ps_shift = c.ps_shift;
    p.max_pages = c.max_pages;
    p.causal = causal;
    p.scale_log2 = scale * kLog2e;
    const unsigned blocks = (unsigned)(B * H * Nq);
    count_launch();
    if (c.d == 128) {
        if (c.scales)
            fa_decode_paged_kernel<128, true><<<blocks, kWarps * 32, 0, stream>>>(p);
        else
            fa_decode_paged_kernel<128, false><<<blocks, kWarps * 32, 0, stream>>>(p);
    } else {
        if (c.scales)
            fa_decode_paged_kernel<64, true><<<blocks, kWarps * 32, 0, stream>>>(p);
        else
            fa_decode_paged_kernel<64, false><<<blocks, kWarps * 32, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace fa
