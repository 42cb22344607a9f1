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
// which find their sequence by bisection in shared memory, four at a time (30K pages
// given and taken back: 10.9 us one by one, 10.1 together).  A slot is taken from the
// stack where its page is new, so no thread waits for a table entry that another
// writes.  Few pages and rows are one block's work (a step of 64 sequences, reserve
// and release: 5.6 us, with eight blocks 7.2).  A map of many rows, and the pages that
// come with it, are dealt out over the whole GPU by a second kernel.
#include <cuda_runtime.h>

#include <atomic>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kMaxSeqs = 4096;        // of one call: their scans lie in shared memory
constexpr int kTablesCluster = 8;
constexpr int kOneBlock = 1 << 15;    // pages and rows that may be one block's work
constexpr int kMapRows = 1 << 16;     // rows up to which the first kernel makes the map
constexpr int kUnroll = 4;

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
    int w = lane < (int)(blockDim.x >> 5) ? part[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += y;
    }
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return warp ? x + before : x;
}

// The last b in [lo, hi] with at[b] <= x (at[lo] <= x, never falling).
__device__ __forceinline__ int last_at(const int* at, int lo, int hi, int x) {
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// What a block knows of all sequences once it has scanned them.
struct Scanned {
    int* len_of;                      // [B] tokens before
    int* page0;                       // [B + 1] pages that the sequences before it need
    int* row0;                        // [B + 1] new tokens of the sequences before it
    int total, n_free;                // pages given away; free pages before
};

__device__ __forceinline__ int pages_of(const TablesParams& p, int tokens) {
    return (tokens + (1 << p.ps_shift) - 1) >> p.ps_shift;
}

// The pages given away, to their tables; thread `at` of `n`.
__device__ __forceinline__ void deal_pages(const TablesParams& p, const Scanned& s, int at, int n) {
#pragma unroll 1
    for (int i0 = at; i0 < s.total; i0 += kUnroll * n) {
        int page[kUnroll];
        long long to[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * n;
            to[u] = -1;
            if (i >= s.total) continue;
            page[u] = p.free_pages[s.n_free - 1 - i];
            const int b = last_at(s.page0, 0, p.B - 1, i);
            to[u] = (long long)b * p.max_pages + pages_of(p, s.len_of[b]) + (i - s.page0[b]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u] >= 0) p.table[to[u]] = page[u];
    }
}

// Positions and slots of the new tokens; thread `at` of `n`.
__device__ __forceinline__ void map_rows(const TablesParams& p, const Scanned& s, int at, int n) {
#pragma unroll 1
    for (long long r0 = at; r0 < p.rows; r0 += kUnroll * n) {
        int pos[kUnroll], page[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long r = r0 + u * n;
            pos[u] = 0;
            page[u] = -1;
            if (r >= p.rows) continue;
            int b, i;
            if (p.N) {
                b = (int)r / p.N;
                i = (int)r - b * p.N;
            } else {
                b = last_at(s.row0, 0, p.B - 1, (int)r);
                i = (int)r - s.row0[b];
            }
            if (i < s.row0[b + 1] - s.row0[b]) {
                pos[u] = s.len_of[b] + i;
                const int j = pos[u] >> p.ps_shift, old = pages_of(p, s.len_of[b]);
                page[u] = j < old ? p.table[(long long)b * p.max_pages + j]
                                  : p.free_pages[s.n_free - 1 - (s.page0[b] + j - old)];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long r = r0 + u * n;
            if (r >= p.rows) continue;
            p.positions[r] = pos[u];
            p.slots[r] = page[u] < 0 ? -1
                                     : ((long long)page[u] << p.ps_shift) +
                                           (pos[u] & ((1 << p.ps_shift) - 1));
        }
    }
}

// ALONE: pages and rows are dealt out here, too (else by fa_kv_fill_kernel).
__global__ void __launch_bounds__(kMostThreads)
fa_kv_reserve_kernel(const __grid_constant__ TablesParams p, bool alone) {
    extern __shared__ int seqs[];                 // [3][B + 1]
    __shared__ int part[2][32], total_sh;
    Scanned s{seqs, seqs + p.B + 1, seqs + 2 * (p.B + 1), 0, 0};
    const int tid = threadIdx.x, nt = blockDim.x;
    const int rank = cluster_rank(), ctas = gridDim.x;    // one cluster
    pdl_wait();
    pdl_launch_dependents();
    s.n_free = min(max(*p.n_free, 0), p.n_pages);
    if (tid == 0) total_sh = 0;
    const int most = p.max_pages << p.ps_shift;
    int pages = 0, rows = 0;                      // of the sequences of the passes before
    for (int base = 0; base < p.B; base += nt) {
        const int b = base + tid;
        int len = 0, n = 0, need = 0;
        if (b < p.B) {
            len = min(max(p.lens[b], 0), most);
            n = max(p.wanted[b], 0);
            if (n > most - len) n = -1;           // its table does not hold them
            else need = pages_of(p, len + n) - pages_of(p, len);
        }
        const int upto = pages + block_scan(need, part[0]);
        const bool served = n >= 0 && (need == 0 || upto <= s.n_free);
        const int count = served ? n : 0;
        const int row_end = rows + block_scan(count, part[1]);
        if (b < p.B) {
            s.len_of[b] = len;
            s.page0[b] = upto - need;
            s.row0[b] = row_end - count;
            if (need > 0 && served) atomicMax(&total_sh, upto);
            if (rank == 0) {
                p.starts[b] = len;
                p.counts[b] = count;
                p.cu[b + 1] = row_end;
            }
        }
        if (tid == nt - 1) {                      // the rounds' sums, for the next round
            s.row0[p.B] = row_end;
            s.page0[p.B] = upto;
        }
        __syncthreads();
        pages = s.page0[p.B];
        rows = s.row0[p.B];
        __syncthreads();
    }
    s.total = total_sh;
    if (ctas > 1) cluster_sync();                 // everybody has read the lengths
    if (rank == 0) {
        for (int b = tid; b < p.B; b += nt) p.lens[b] = s.len_of[b] + (s.row0[b + 1] - s.row0[b]);
        if (tid == 0) {
            *p.n_free = s.n_free - s.total;
            p.cu[0] = 0;
        }
    }
    if (!alone) return;
    deal_pages(p, s, rank * nt + tid, ctas * nt);
    if (p.slots) map_rows(p, s, rank * nt + tid, ctas * nt);
}

// The second part of a call with a large map: each block scans the pages that were
// given (from starts and counts) for itself.
__global__ void __launch_bounds__(kMostThreads)
fa_kv_fill_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int seqs[];
    __shared__ int part[32];
    Scanned s{seqs, seqs + p.B + 1, seqs + 2 * (p.B + 1), 0, 0};
    const int tid = threadIdx.x, nt = blockDim.x;
    pdl_wait();
    pdl_launch_dependents();
    const int left = *p.n_free;
    if (tid == 0) s.row0[0] = 0;
    for (int base = 0; base < p.B; base += nt) {
        const int b = base + tid;
        int len = 0, given = 0;
        if (b < p.B) {
            len = p.starts[b];
            given = pages_of(p, len + p.counts[b]) - pages_of(p, len);
            s.len_of[b] = len;
            s.row0[b + 1] = p.cu[b + 1];
        }
        const int upto = s.total + block_scan(given, part);
        if (b < p.B) s.page0[b] = upto - given;
        if (tid == nt - 1) s.page0[p.B] = upto;
        __syncthreads();
        s.total = s.page0[p.B];
        __syncthreads();
    }
    s.n_free = left + s.total;
    deal_pages(p, s, blockIdx.x * nt + tid, gridDim.x * nt);
    map_rows(p, s, blockIdx.x * nt + tid, gridDim.x * nt);
}

__global__ void __launch_bounds__(kMostThreads)
fa_kv_release_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int seqs[];                 // [2][B + 1]
    int* const from = seqs;                       // first page that is given back
    int* const page0 = seqs + p.B + 1;            // pages that the sequences before it give back
    __shared__ int part[32];
    const int tid = threadIdx.x, nt = blockDim.x;
    const int rank = cluster_rank(), ctas = gridDim.x;
    pdl_wait();
    pdl_launch_dependents();
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    const int most = p.max_pages << p.ps_shift;
    auto kept = [&](int b, int len) { return min(len, max(p.wanted[b], 0)); };
    int pages = 0;
    for (int base = 0; base < p.B; base += nt) {
        const int b = base + tid;
        int gone = 0, first = 0;
        if (b < p.B) {
            const int len = min(max(p.lens[b], 0), most);
            const int last = pages_of(p, len);
            first = pages_of(p, kept(b, len));
            if (p.pinned) first = min(last, max(first, p.pinned[b]));
            gone = last - first;
        }
        const int upto = pages + block_scan(gone, part);
        if (b < p.B) {
            from[b] = first;
            page0[b] = upto - gone;
        }
        if (tid == nt - 1) page0[p.B] = upto;
        __syncthreads();
        pages = page0[p.B];
        __syncthreads();
    }
    if (ctas > 1) cluster_sync();                 // everybody has read the lengths
    if (rank == 0) {
        for (int b = tid; b < p.B; b += nt) {
            const int len = min(max(p.lens[b], 0), most), keep = kept(b, len);
            p.lens[b] = keep;
            // pinned pages behind the kept tokens leave the table and stay taken
            for (int j = pages_of(p, keep); j < from[b]; ++j)
                p.table[(long long)b * p.max_pages + j] = -1;
        }
        if (tid == 0) *p.n_free = min(n_free + pages, p.n_pages);
    }
#pragma unroll 1
    for (int i0 = rank * nt + tid; i0 < pages; i0 += kUnroll * ctas * nt) {
        int* entry[kUnroll];
        int page[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * ctas * nt;
            entry[u] = nullptr;
            if (i >= pages) continue;
            const int b = last_at(page0, 0, p.B - 1, i);
            entry[u] = p.table + (long long)b * p.max_pages + from[b] + (i - page0[b]);
            page[u] = *entry[u];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * ctas * nt;
            if (!entry[u]) continue;
            if (n_free + i < p.n_pages) p.free_pages[n_free + i] = page[u];
            *entry[u] = -1;
        }
    }
}

// The map of rows whose table is already there.  A block's rows lie in few sequences:
// those of its first and its last row are found once, a row's between them.
__global__ void __launch_bounds__(256)
fa_kv_slots_kernel(const __grid_constant__ TablesParams p) {
    __shared__ int ends[2];
    pdl_wait();
    pdl_launch_dependents();
    const long long first = (long long)blockIdx.x * (256 * kUnroll);
    if (!p.N) {
        if (threadIdx.x == 0) ends[0] = last_at(p.cu, 0, p.B - 1, (int)first);
        if (threadIdx.x == 32)
            ends[1] = last_at(p.cu, 0, p.B - 1,
                              (int)min(first + 256 * kUnroll - 1, (long long)p.rows - 1));
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const long long r = first + u * 256 + threadIdx.x;
        if (r >= p.rows) return;
        int b, i, n;
        if (p.N) {
            b = (int)r / p.N;
            i = (int)r - b * p.N;
            n = p.counts[b];
        } else {
            // (offsets that fall somewhere: any b of the two is inside)
            b = last_at(p.cu, ends[0], max(ends[0], ends[1]), (int)r);
            i = (int)r - p.cu[b];
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
}

// Once a device: the shared memory that the kernels may use.
cudaError_t configure() {
    static std::atomic<unsigned long long> configured{0};     // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || ((configured.load(std::memory_order_acquire) >> dev) & 1)) return e;
    const int bytes = 3 * (kMaxSeqs + 1) * (int)sizeof(int);
    for (const void* kernel : {(const void*)fa_kv_reserve_kernel, (const void*)fa_kv_fill_kernel,
                               (const void*)fa_kv_release_kernel})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) configured.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

cudaError_t launch_slots(const TablesParams& p, cudaStream_t stream) {
    constexpr long long per = 256 * kUnroll;
    return launch_pdl(fa_kv_slots_kernel, (unsigned)((p.rows + per - 1) / per), 256, 0, 1, stream,
                      p);
}

// Threads of a block: a warp for every 32 sequences, and enough of them for the rest.
unsigned threads_for(int B, bool one) { return one && B <= 256 ? 256 : kMostThreads; }

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
    const TablesParams p{block_table, seqlens, free_pages, n_free, new_tokens, nullptr, starts,
                         counts, cu_seqlens, positions, slots, B, N, (int)rows, n_pages,
                         shift_of(page_size), max_pages};
    const size_t smem = 3 * (B + 1) * sizeof(int);
    const bool alone = rows <= kMapRows;
    // pages that the call may give away: with a packed map those of its rows
    const long long most = (rows && !N ? rows / page_size + B : (long long)B * max_pages) + rows;
    const bool one = !alone || most <= kOneBlock;
    const int ctas = one ? 1 : kTablesCluster;
    cudaError_t e = launch_pdl(fa_kv_reserve_kernel, ctas, threads_for(B, one), smem, ctas,
                               (cudaStream_t)stream, p, alone);
    if (e == cudaSuccess && !alone) {
        // two blocks an SM: 6.8 us for the map of 540K rows, 7.0 with one of 1024 threads
        const unsigned sms = device_sm_count() > 0 ? device_sm_count() : 152;
        e = launch_pdl(fa_kv_fill_kernel, 2 * sms, 512, smem, 1, (cudaStream_t)stream, p);
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
    const bool one = (long long)B * max_pages <= kOneBlock;
    const int ctas = one ? 1 : kTablesCluster;
    const cudaError_t e = launch_pdl(fa_kv_release_kernel, ctas, threads_for(B, one),
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
