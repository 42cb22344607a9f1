// What the dK/dV kernels of the backward with keys of another length share: their
// parameters, the work items, and the constant operand of the extension MMAs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

constexpr int kBwdKeys = 128;   // keys per work item

struct BwdParams {
    int H, Hkv, N, Np, G, causal;
    int rows;                         // rows per head of q: N, or the packed total
    // Packed: sequence b's queries are rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of every
    // head; N is then the longest sequence and the workspace keeps N-row (padded) regions
    // per (batch, head).
    const int* cu_seqlens;
    // At most Nk keys a sequence, krows rows a head of k, v, dk, dv.  Padded batches:
    // kv_lens[b] keys, or Nk (null); packed ones: rows cu_k[b] .. cu_k[b + 1] - 1.
    int Nk, krows;
    const int* kv_lens;
    const int* cu_k;
    float scale, scale_log2;
    const uint16_t* lse_ext;          // workspace tables (fa_internal.h)
    const uint16_t* d_ext;
    float* dq_acc;
    int* work;                        // next work item (zero on entry, left zero)
    int n_bg, n_items;                // B * Hkv; work items (B * Hkv * key blocks)
    __nv_bfloat16* dk;
    __nv_bfloat16* dv;
    DeviceStatus* status;
};

inline BwdParams bwd_params(const Shape& s, void* dk, void* dv, const BwdWorkspace& ws,
                            DeviceStatus* status) {
    const bool packed = s.cu_seqlens != nullptr;
    BwdParams p;
    p.H = s.H;
    p.Hkv = s.Hkv;
    p.N = s.N;
    p.Np = padded_rows(s.N);
    p.G = s.H / s.Hkv;
    p.causal = s.causal;
    p.rows = packed ? s.total : s.N;
    p.cu_seqlens = s.cu_seqlens;
    p.Nk = s.Nk;
    p.krows = packed ? s.total_k : s.Nk;
    p.kv_lens = s.kv_lens;
    p.cu_k = s.cu_k;
    p.scale = s.scale;
    p.scale_log2 = (float)((double)s.scale * 1.4426950408889634);
    p.lse_ext = ws.lse_ext;
    p.d_ext = ws.d_ext;
    p.dq_acc = ws.dq_acc;
    p.work = ws.work;
    p.n_bg = s.B * s.Hkv;
    p.n_items = (s.Nk + kBwdKeys - 1) / kBwdKeys * p.n_bg;
    p.dk = static_cast<__nv_bfloat16*>(dk);
    p.dv = static_cast<__nv_bfloat16*>(dv);
    p.status = status;
    return p;
}

// What one dK/dV work item covers: kv head bg = b * Hkv + g, key block jblk, and the range of
// query blocks (of br rows) that see some key of the block.
struct BwdCta {
    int jblk, b, g, bg, z_kv, i_start, n_i, n_it;
    int tok0, q_len;     // first query row of the sequence in its head, and their number
    int ktok0, seq_len;  // the same of its keys
    int off;             // query i sees keys j <= i + off under the causal mask
    bool idle;           // a key block past its sequence's end: nothing to do
};
__device__ __forceinline__ BwdCta bwd_cta(const BwdParams& p, int br, int bg, int jblk) {
    BwdCta c;
    const bool packed = p.cu_seqlens != nullptr;
    c.bg = bg;
    c.jblk = jblk;
    c.b = bg / p.Hkv;
    c.g = bg - c.b * p.Hkv;
    c.tok0 = c.ktok0 = 0;
    c.q_len = packed ? packed_seq(p.cu_seqlens, c.b, p.N, p.rows, c.tok0) : p.N;
    c.seq_len = packed      ? packed_seq(p.cu_k, c.b, p.Nk, p.krows, c.ktok0)
                : p.kv_lens ? min(max(__ldg(p.kv_lens + c.b), 0), p.Nk)
                            : p.Nk;
    c.off = c.seq_len - c.q_len;
    c.idle = jblk * kBwdKeys >= c.seq_len;
    c.z_kv = packed ? c.g : bg;
    const int n_qblk = (c.q_len + br - 1) / br;
    c.i_start = p.causal ? max(0, jblk * kBwdKeys - c.off) / br : 0;
    c.n_i = max(0, n_qblk - c.i_start);
    c.n_it = p.G * c.n_i;
    return c;
}

// The constant A operand of the extension MMAs, 128 key rows x 16 columns:
// cols 0-8 hold 1/c as three bf16 terms (h h h m m m l l l), against the B
// columns (x_h x_m x_l) x 3 of -LSE log2(e), so that the nine products sum to
// (-LSE log2 e) / c; cols 9-11 hold 1 against the three terms of -D; the rest
// 0.  One 16-byte piece per thread of the first 256.
__device__ __forceinline__ void bwd_fill_ones(uint8_t* sOnes, float scale_log2) {
    if (threadIdx.x < kBwdKeys * 32 / 16) {
        const float inv = 1.0f / scale_log2;
        const float ih = bf16_round(inv), im = bf16_round(inv - ih),
                    il = bf16_round(inv - ih - im);
        const int kc = (threadIdx.x >> 3) & 1;   // K half of this core-matrix row
        uint4 w;
        if (kc == 0) {
            w.x = pack_bf16x2(ih, ih);
            w.y = pack_bf16x2(ih, im);
            w.z = pack_bf16x2(im, im);
            w.w = pack_bf16x2(il, il);
        } else {
            w.x = pack_bf16x2(il, 1.0f);
            w.y = pack_bf16x2(1.0f, 1.0f);
            w.z = 0u;
            w.w = 0u;
        }
        *reinterpret_cast<uint4*>(sOnes + threadIdx.x * 16) = w;
        fence_proxy_async_smem();
    }
}

// Clears rows [from, rows) of a tile of `chunks` 128-byte-wide swizzled chunks, one row
// a thread and turn, threads t of n.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int chunks, int rows, int from, int t,
                                           int n) {
    for (int r = max(from, 0) + t; r < rows; r += n)
        for (int c = 0; c < chunks; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
                *reinterpret_cast<uint4*>(tile + c * (rows * 128) + r * 128 + u * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
}

// Zeros in dK and dV (columns [c_lo, c_hi) of this thread's key row) of a key block that
// no query sees or that lies past a padded sequence's keys.
template <int D>
__device__ __forceinline__ void zero_grads(const BwdParams& p, const BwdCta& c, int key, int c_lo,
                                           int c_hi, bool dk, bool dv) {
    if (key >= (p.cu_seqlens ? c.seq_len : p.Nk)) return;
    const size_t row = ((size_t)c.z_kv * p.krows + c.ktok0 + key) * D;
    for (int e = c_lo; e < c_hi; e += 8) {
        if (dk) *reinterpret_cast<uint4*>(p.dk + row + e) = make_uint4(0u, 0u, 0u, 0u);
        if (dv) *reinterpret_cast<uint4*>(p.dv + row + e) = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace fa
