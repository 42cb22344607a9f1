// Block tables and slot maps of the paged key/value cache, kept on the GPU: pages
// given to requests in their order, the position and the slot (page * page_size +
// row) of every new token, and pages taken back.
//
// The free pages are a stack: free_pages[0 .. n_free - 1].  With len_b tokens in
// the cache and n_b more to come, sequence b needs
//     need_b = ceil((len_b + n_b) / page_size) - ceil(len_b / page_size)
// pages more, and is served iff its table holds them and need_b = 0 or the sum of
// the needs up to and with it is at most n_free.  That sum never falls, so of the
// sequences that need pages a prefix is served, and page i of those given away
// (in the order of the sequences, then of their pages) is free_pages[n_free - 1 - i].
//
// The numbers a sequence has are a few ints, so the calls are bound by their launch
// and by the two scans over the sequences; one launch does all of it.  Every block
// of a cluster scans all sequences for itself (no block waits for a result of
// another), the cluster's barrier stands between the last read of the lengths and
// their update in place, and pages and rows are dealt out over the cluster's threads,
// which find their sequence by bisection in shared memory.  A slot is taken from the
// stack where its page is new, so no thread waits for a table entry that another
// writes.
#include <cuda_runtime.h>

#include <atomic>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxSeqs = 4096;        // of one call: their scans lie in shared memory
constexpr int kTablesCluster = 8;

struct TablesParams {
    int* table;
    int* lens;
    int* free_pages;
    int* n_free;
    const int* wanted;                // reserve: new tokens; release: tokens to keep
    const int* pinned;                // release: first pages that are not given back, or null
    int* starts;
    int* counts;
    int* cu;
    int* positions;                   // null: no map
    long long* slots;
    int B, N, rows, n_pages, ps_shift, max_pages;   // N: rows a sequence, 0 = packed
};

// Inclusive sum over the block's threads; `part` is 32 ints of shared memory that
// nobody uses before the block's next barrier but one.
__device__ __forceinline__ int block_scan(int x, int* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int w = part[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return warp ? x + before : x;
}

// The last b < n with at[b] <= x (at[0] <= x, never falling).
__device__ __forceinline__ int last_at(const int* at, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads)
fa_kv_reserve_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int seqs[];                 // [3][B + 1]
    int* const len_of = seqs;                     // tokens before
    int* const page0 = seqs + p.B + 1;            // pages that the sequences before it need
    int* const row0 = page0 + p.B + 1;            // rows of the sequences before it
    __shared__ int part[2][32], total_sh;
    const int tid = threadIdx.x, ps_mask = (1 << p.ps_shift) - 1;
    const int rank = cluster_rank(), ctas = gridDim.x;    // one cluster
    pdl_wait();
    pdl_launch_dependents();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    if (tid == 0) total_sh = 0;
    const int most = p.max_pages << p.ps_shift;
    int pages = 0, rows = 0;                      // of the sequences before this round's
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        int len = 0, n = 0, need = 0;
        if (b < p.B) {
            len = min(max(p.lens[b], 0), most);
            n = max(p.wanted[b], 0);
            if (n > most - len) n = -1;           // its table does not hold them
            else need = ((len + n + ps_mask) >> p.ps_shift) - ((len + ps_mask) >> p.ps_shift);
        }
        const int upto = pages + block_scan(need, part[0]);
        const bool served = n >= 0 && (need == 0 || upto <= n_free);
        const int count = served ? n : 0;
        const int row_end = rows + block_scan(count, part[1]);
        if (b < p.B) {
            len_of[b] = len;
            page0[b] = upto - need;
            row0[b] = row_end - count;
            if (need > 0 && served) atomicMax(&total_sh, upto);
            if (rank == 0) {
                p.starts[b] = len;
                p.counts[b] = count;
                p.cu[b + 1] = row_end;
            }
        }
        if (tid == kThreads - 1) {                // the rounds' sums, for the next round
            row0[p.B] = row_end;
            page0[p.B] = upto;
        }
        __syncthreads();
        pages = page0[p.B];
        rows = row0[p.B];
        __syncthreads();
    }
    const int total = total_sh;
    if (ctas > 1) cluster_sync();                 // everybody has read the lengths
    if (rank == 0) {
        for (int b = tid; b < p.B; b += kThreads) p.lens[b] = len_of[b] + (row0[b + 1] - row0[b]);
        if (tid == 0) {
            *p.n_free = n_free - total;
            p.cu[0] = 0;
        }
    }
    auto have = [&](int b) { return (len_of[b] + ps_mask) >> p.ps_shift; };
    for (int i = rank * kThreads + tid; i < total; i += ctas * kThreads) {
        const int b = last_at(page0, p.B, i);
        p.table[(long long)b * p.max_pages + have(b) + (i - page0[b])] =
            p.free_pages[n_free - 1 - i];
    }
    if (!p.slots) return;
    for (int r = rank * kThreads + tid; r < p.rows; r += ctas * kThreads) {
        int b, i;
        if (p.N) {
            b = r / p.N;
            i = r - b * p.N;
        } else {
            b = last_at(row0, p.B, r);
            i = r - row0[b];
        }
        int pos = 0;
        long long slot = -1;
        if (i < row0[b + 1] - row0[b]) {
            pos = len_of[b] + i;
            const int j = pos >> p.ps_shift, old = have(b);
            const int page = j < old ? p.table[(long long)b * p.max_pages + j]
                                     : p.free_pages[n_free - 1 - (page0[b] + j - old)];
            if (page >= 0) slot = ((long long)page << p.ps_shift) + (pos & ps_mask);
        }
        p.positions[r] = pos;
        p.slots[r] = slot;
    }
}

__global__ void __launch_bounds__(kThreads)
fa_kv_release_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int seqs[];                 // [2][B + 1]
    int* const from = seqs;                       // first page that is given back
    int* const page0 = seqs + p.B + 1;            // pages that the sequences before it give back
    __shared__ int part[32];
    const int tid = threadIdx.x, ps_mask = (1 << p.ps_shift) - 1;
    const int rank = cluster_rank(), ctas = gridDim.x;
    pdl_wait();
    pdl_launch_dependents();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    const int most = p.max_pages << p.ps_shift;
    auto kept = [&](int b, int len) { return min(len, max(p.wanted[b], 0)); };
    int pages = 0;
    for (int base = 0; base < p.B; base += kThreads) {
        const int b = base + tid;
        int gone = 0, first = 0;
        if (b < p.B) {
            const int len = min(max(p.lens[b], 0), most);
            const int last = (len + ps_mask) >> p.ps_shift;
            first = (kept(b, len) + ps_mask) >> p.ps_shift;
            if (p.pinned) first = min(last, max(first, p.pinned[b]));
            gone = last - first;
        }
        const int upto = pages + block_scan(gone, part);
        if (b < p.B) {
            from[b] = first;
            page0[b] = upto - gone;
        }
        if (tid == kThreads - 1) page0[p.B] = upto;
        __syncthreads();
        pages = page0[p.B];
        __syncthreads();
    }
    if (ctas > 1) cluster_sync();                 // everybody has read the lengths
    if (rank == 0) {
        for (int b = tid; b < p.B; b += kThreads) {
            const int len = min(max(p.lens[b], 0), most), keep = kept(b, len);
            p.lens[b] = keep;
            // pinned pages behind the kept tokens leave the table and stay taken
            for (int j = (keep + ps_mask) >> p.ps_shift; j < from[b]; ++j)
                p.table[(long long)b * p.max_pages + j] = -1;
        }
        if (tid == 0) *p.n_free = min(n_free + pages, p.n_pages);
    }
    for (int i = rank * kThreads + tid; i < pages; i += ctas * kThreads) {
        const int b = last_at(page0, p.B, i);
        int* const entry = p.table + (long long)b * p.max_pages + from[b] + (i - page0[b]);
        if (n_free + i < p.n_pages) p.free_pages[n_free + i] = *entry;
        *entry = -1;
    }
}

// The map of rows whose table is already there.
__global__ void __launch_bounds__(256)
fa_kv_slots_kernel(const __grid_constant__ TablesParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= p.rows) return;
    int b, i, n;
    if (p.N) {
        b = r / p.N;
        i = r - b * p.N;
        n = p.counts[b];
    } else {
        b = last_at(p.cu, p.B, r);
        i = r - p.cu[b];
        n = p.cu[b + 1] - p.cu[b];
    }
    long long pos = (long long)p.starts[b] + i, slot = -1;
    if (i >= 0 && i < n && pos >= 0 && (pos >> p.ps_shift) < p.max_pages) {
        const int page = p.table[(long long)b * p.max_pages + (pos >> p.ps_shift)];
        if (page >= 0)
            slot = ((long long)page << p.ps_shift) + (pos & ((1 << p.ps_shift) - 1));
    } else {
        pos = 0;
    }
    p.positions[r] = (int)pos;
    p.slots[r] = slot;
}

// Once a device: the shared memory that the two kernels may use.
cudaError_t configure() {
    static std::atomic<unsigned long long> configured{0};     // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || ((configured.load(std::memory_order_acquire) >> dev) & 1)) return e;
    const int bytes = 3 * (kMaxSeqs + 1) * (int)sizeof(int);
    e = cudaFuncSetAttribute(fa_kv_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fa_kv_release_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 bytes);
    if (e == cudaSuccess) configured.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

cudaError_t launch_slots(const TablesParams& p, cudaStream_t stream) {
    return launch_pdl(fa_kv_slots_kernel, (unsigned)((p.rows + 255LL) / 256), 256, 0, 1, stream, p);
}

// Rows up to which the map is made by the launch that gives the pages.
constexpr int kMapRows = 1 << 16;

fa_status check_ints(const void* p) { return check_pointer(p, alignof(int)); }

fa_status check_table_shape(int B, long long n_pages, int page_size, int max_pages) {
    if (B < 1 || n_pages < 1 || page_size < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
        return FA_ERR_UNSUPPORTED;
    if ((long long)max_pages * page_size >= (1LL << 30) || (long long)B * max_pages >= (1LL << 30) ||
        (n_pages + B) * page_size >= (1LL << 31))
        return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_kv_reserve(int* block_table, int* seqlens, int* free_pages, int* n_free,
                        const int* new_tokens, int* starts, int* counts, int* cu_seqlens,
                        int* positions, long long* slots, int B, int N, int total, int n_pages,
                        int page_size, int max_pages, fa_stream_t stream) {
    fa_status st = check_table_shape(B, n_pages, page_size, max_pages);
    for (const void* x : {(const void*)block_table, (const void*)seqlens, (const void*)free_pages,
                          (const void*)n_free, (const void*)new_tokens, (const void*)starts,
                          (const void*)counts, (const void*)cu_seqlens})
        if (st == FA_OK) st = check_ints(x);
    if (st != FA_OK) return st;
    if (B > kMaxSeqs) return FA_ERR_UNSUPPORTED;
    long long rows = 0;
    if (positions || slots) {
        if ((st = check_ints(positions)) != FA_OK ||
            (st = check_pointer(slots, alignof(long long))) != FA_OK)
            return st;
        if (N < 0 || (N == 0 && total < 1)) return FA_ERR_INVALID_ARG;
        rows = N ? (long long)B * N : total;
        if (rows >= (1LL << 31) - (1 << 16)) return FA_ERR_UNSUPPORTED;
    }
    int dev;
    DeviceStatus* status;
    if ((st = ready_device(&dev, &status)) != FA_OK) return st;
    if (configure() != cudaSuccess) return FA_ERR_CUDA;
    const bool apart = rows > kMapRows;
    TablesParams p{block_table, seqlens, free_pages, n_free, new_tokens, nullptr, starts, counts,
                   cu_seqlens, positions, apart ? nullptr : slots, B, N, (int)rows, n_pages,
                   shift_of(page_size), max_pages};
    const int ctas = kTablesCluster;
    cudaError_t e = launch_pdl(fa_kv_reserve_kernel, ctas, kThreads,
                               3 * (B + 1) * sizeof(int), ctas, (cudaStream_t)stream, p);
    if (e == cudaSuccess && apart) {
        p.slots = slots;
        e = launch_slots(p, (cudaStream_t)stream);
    }
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_kv_release(int* block_table, int* seqlens, int* free_pages, int* n_free,
                        const int* keep, const int* pinned, int B, int n_pages, int page_size,
                        int max_pages, fa_stream_t stream) {
    fa_status st = check_table_shape(B, n_pages, page_size, max_pages);
    for (const void* x : {(const void*)block_table, (const void*)seqlens, (const void*)free_pages,
                          (const void*)n_free, (const void*)keep})
        if (st == FA_OK) st = check_ints(x);
    if (st == FA_OK && pinned) st = check_ints(pinned);
    if (st != FA_OK) return st;
    if (B > kMaxSeqs) return FA_ERR_UNSUPPORTED;
    int dev;
    DeviceStatus* status;
    if ((st = ready_device(&dev, &status)) != FA_OK) return st;
    if (configure() != cudaSuccess) return FA_ERR_CUDA;
    const TablesParams p{block_table, seqlens, free_pages, n_free, keep, pinned, nullptr, nullptr,
                         nullptr, nullptr, nullptr, B, 0, 0, n_pages, shift_of(page_size),
                         max_pages};
    const int ctas = kTablesCluster;
    const cudaError_t e = launch_pdl(fa_kv_release_kernel, ctas, kThreads,
                                     2 * (B + 1) * sizeof(int), ctas, (cudaStream_t)stream, p);
    return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

static fa_status slots_of(const int* block_table, const int* starts, const int* counts,
                          const int* cu_seqlens, int* positions, long long* slots, int B, int N,
                          long long rows, int page_size, int max_pages, fa_stream_t stream) {
    fa_status st = check_table_shape(B, 1, page_size, max_pages);
    for (const void* x : {(const void*)block_table, (const void*)starts,
                          (const void*)(N ? counts : cu_seqlens), (const void*)positions})
        if (st == FA_OK) st = check_ints(x);
    if (st == FA_OK) st = check_pointer(slots, alignof(long long));
    if (st != FA_OK) return st;
    if (rows >= (1LL << 31) - (1 << 16)) return FA_ERR_UNSUPPORTED;
    int dev;
    DeviceStatus* status;
    if ((st = ready_device(&dev, &status)) != FA_OK) return st;
    const TablesParams p{const_cast<int*>(block_table), nullptr, nullptr, nullptr, nullptr, nullptr,
                         const_cast<int*>(starts), const_cast<int*>(counts),
                         const_cast<int*>(cu_seqlens), positions, slots, B, N, (int)rows, 1,
                         shift_of(page_size), max_pages};
    return launch_slots(p, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_kv_slots(const int* block_table, const int* starts, const int* counts, int* positions,
                      long long* slots, int B, int N, int page_size, int max_pages,
                      fa_stream_t stream) {
    if (N < 1) return FA_ERR_INVALID_ARG;
    return slots_of(block_table, starts, counts, nullptr, positions, slots, B, N, (long long)B * N,
                    page_size, max_pages, stream);
}

fa_status fa_kv_slots_varlen(const int* block_table, const int* starts, const int* cu_seqlens,
                             int* positions, long long* slots, int B, int total, int page_size,
                             int max_pages, fa_stream_t stream) {
    if (total < 1) return FA_ERR_INVALID_ARG;
    return slots_of(block_table, starts, nullptr, cu_seqlens, positions, slots, B, 0, total,
                    page_size, max_pages, stream);
}

}  // extern "C"
