// Before and after the dK/dV pass of the backward with keys of another length: the tables of
// -LSE log2(e) and -D = -rowsum(dO o O) with a zeroed dQ accumulator, and at d = 128 the
// accumulator rounded to dQ (at d = 64 that kernel is beside its dK/dV pass, whose order of
// columns it knows).  Rows and layouts are those of fa_bwd.cu's kernels, which go through all
// rows with a 64-bit division and a chain of dependent loads each.  Here a block has 32 to 128
// rows of one head, finds its sequence once and has four rows' loads a thread in flight:
// 16 packed sequences of 128 to 1024 queries, H32, d = 128, 74 and 48 us there, 47 and 28 here;
// bound by HBM.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "bwd_parts.cuh"

namespace fa {
namespace {

constexpr int kPasses = 4;

// The queries of one head: how many, and the first one's row in q.
__device__ __forceinline__ int query_rows(const BwdParams& p, int bh, long long& base) {
    base = (long long)bh * p.N;
    if (!p.cu_seqlens) return p.N;
    int t0;
    const int b = bh / p.H, len = packed_seq(p.cu_seqlens, b, p.N, p.rows, t0);
    base = (long long)(bh - b * p.H) * p.rows + t0;
    return len;
}

// D / 8 lanes a row.  Rows past the sequence, up to a multiple of 128, are read by the next
// kernel: -1e30 for their LSE, so that P = 0, as for a row that sees no key (LSE = -infinity).
template <int D>
__global__ void __launch_bounds__(256)
cross_pre_kernel(const __nv_bfloat16* __restrict__ o, const __nv_bfloat16* __restrict__ dout,
                 const float* __restrict__ lse, uint16_t* __restrict__ lse_ext,
                 uint16_t* __restrict__ d_ext, const BwdParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, kStep = 8 * RPW, kRows = kStep * kPasses;
    static_assert(kRowPad % kRows == 0, "a block is read as a whole, or not at all");
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.work = 0;
    const int n_blk = p.Np / kRows, bh = (int)blockIdx.x / n_blk;
    const int r0 = ((int)blockIdx.x - bh * n_blk) * kRows;
    long long base;
    const int len = query_rows(p, bh, base);
    if (r0 >= (len + kRowPad - 1) / kRowPad * kRowPad) return;
    const long long acc_row = (long long)bh * p.Np + r0;
    float4* const z = reinterpret_cast<float4*>(p.dq_acc + acc_row * D);
#pragma unroll
    for (int e = 0; e < kRows * D / 4 / 256; ++e)
        z[e * 256 + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int lane = threadIdx.x & 31, sl = lane % LPR;
    const int at = (threadIdx.x >> 5) * RPW + lane / LPR;
    uint4 x[kPasses], y[kPasses];
    float l[kPasses];
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
        const int i = r0 + s * kStep + at;
        x[s] = y[s] = make_uint4(0u, 0u, 0u, 0u);
        l[s] = CUDART_INF_F;
        if (i < len) {
            x[s] = *reinterpret_cast<const uint4*>(o + (base + i) * D + sl * 8);
            y[s] = *reinterpret_cast<const uint4*>(dout + (base + i) * D + sl * 8);
            if (sl == 0) l[s] = -lse[base + i] * 1.4426950408889634f;
        }
    }
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
        const __nv_bfloat162* const a = reinterpret_cast<const __nv_bfloat162*>(&x[s]);
        const __nv_bfloat162* const b = reinterpret_cast<const __nv_bfloat162*>(&y[s]);
        float d = 0.0f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float2 u = __bfloat1622float2(a[t]), w = __bfloat1622float2(b[t]);
            d = fmaf(u.x, w.x, d);
            d = fmaf(u.y, w.y, d);
        }
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        const long long r = acc_row + s * kStep + at;
        if (sl == 0) write_lse_ext_row(lse_ext, r, l[s] == CUDART_INF_F ? -1e30f : l[s]);
        if (sl == 1) {   // -D in columns 9-11
            const float v = -d;
            const float h = bf16_round(v), m = bf16_round(v - h), w = bf16_round(v - h - m);
            uint16_t* const row = d_ext + ((r >> 3) * 2 * 8 + (r & 7)) * 8;
            *reinterpret_cast<uint4*>(row) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(row + 64) =
                make_uint4(pack_bf16x2(0.0f, h), pack_bf16x2(m, w), 0u, 0u);
        }
    }
}

__global__ void __launch_bounds__(256)
cross_dq128_kernel(__nv_bfloat16* __restrict__ dq, const BwdParams p) {
    constexpr int D = 128, kRows = 8 * kPasses;
    pdl_wait();
    const int joins = p.parts > 1 ? kJoinBlocks * p.n_base : 0;
    if ((int)blockIdx.x < joins) {
        join_parts<D>(p, 64, blockIdx.x);
        return;
    }
    const int n_blk = p.Np / kRows, at = (int)blockIdx.x - joins, bh = at / n_blk;
    const int r0 = (at - bh * n_blk) * kRows;
    long long base;
    const int len = query_rows(p, bh, base);
    const float4* const src =
        reinterpret_cast<const float4*>(p.dq_acc + ((long long)bh * p.Np + r0) * D);
    float4 x[kPasses];
#pragma unroll
    for (int s = 0; s < kPasses; ++s)
        if (r0 + s * 8 + (int)threadIdx.x / 32 < len) x[s] = src[s * 256 + threadIdx.x];
#pragma unroll
    for (int s = 0; s < kPasses; ++s) {
        const int i = r0 + s * 8 + (int)threadIdx.x / 32;
        if (i < len)
            *reinterpret_cast<uint2*>(dq + (base + i) * D + threadIdx.x % 32 * 4) =
                make_uint2(pack_bf16x2(x[s].x * p.scale, x[s].y * p.scale),
                           pack_bf16x2(x[s].z * p.scale, x[s].w * p.scale));
    }
}

}  // namespace

size_t cross_bwd_workspace_bytes(const Shape& s) {
    return bwd_workspace_bytes(s) + bwd_part_bytes(s);
}

cudaError_t launch_bwd_cross_pre(const Shape& s, const void* o, const void* dout, const float* lse,
                                 const BwdWorkspace& ws, cudaStream_t stream) {
    const BwdParams p = bwd_params(s, nullptr, nullptr, ws, nullptr);
    const auto* o_ = static_cast<const __nv_bfloat16*>(o);
    const auto* d_ = static_cast<const __nv_bfloat16*>(dout);
    const unsigned grid = (unsigned)((long long)s.B * s.H * p.Np / (s.d == 128 ? 64 : 128));
    count_launch();
    if (s.d == 128)
        cross_pre_kernel<128><<<grid, 256, 0, stream>>>(o_, d_, lse, ws.lse_ext, ws.d_ext, p);
    else
        cross_pre_kernel<64><<<grid, 256, 0, stream>>>(o_, d_, lse, ws.lse_ext, ws.d_ext, p);
    return cudaGetLastError();
}

cudaError_t launch_bwd_cross_dq128(const Shape& s, const BwdWorkspace& ws, void* dq, void* dk,
                                   void* dv, cudaStream_t stream) {
    const BwdParams p = bwd_params(s, dk, dv, ws, nullptr);
    const unsigned grid = (unsigned)((long long)s.B * s.H * p.Np / (8 * kPasses)) +
                          (p.parts > 1 ? kJoinBlocks * p.n_base : 0);
    return launch_pdl(cross_dq128_kernel, dim3(grid), 256, 0, 1, stream,
                      static_cast<__nv_bfloat16*>(dq), p);
}

}  // namespace fa
