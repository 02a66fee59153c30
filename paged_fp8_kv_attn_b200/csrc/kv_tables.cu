// kv_tables.cu -- page tables and slot maps from request lengths.
//
// Row b grows from o = old_lens[b] to n = new_lens[b] tokens, which takes
// need_b = ceil(n / P) - ceil(o / P) pages.  With U_b = sum_{i <= b} need_i, a
// row is served while U_b fits the free stack; its k-th page is then the
// stack's entry num_free - 1 - (U_b - need_b) - k, its new tokens' slots follow
// from its entries, and the packed position of its first new token is
// sum_{i < b} (n_i - o_i): two prefix sums, then independent work per page
// and per token.
//
// Bound by latency (a decode step moves about 1 KB): one launch of one
// cluster.  Every CTA repeats the prefix sums of all rows, so nothing is
// handed from CTA to CTA, and takes its share of the pages and tokens.
// num_free may be the word that num_free_out names: one CTA writes it after
// the cluster's barrier, when all have read it.
#include "device.cuh"
#include "internal.h"

namespace pkv {

constexpr int kTableThreads = 512;
constexpr int kTableRows = kTableThreads;   // rows whose sums a pass holds in shared memory
constexpr int kTableTokens = 4;             // consecutive tokens a thread takes at a time
constexpr int kTableMaxCluster = 8;

// Sums of non-negative 32-bit numbers, held at 2^31 - 1 (associative, so the
// scan may group them in any way).  Lengths that are no request's cannot wrap.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
    return min(a + b, 0x7FFFFFFFu);
}

// Index of the last of the n (>= 1) non-decreasing values that is <= x; v[0] <= x.
__device__ __forceinline__ int last_at_most(const uint32_t* v, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTableThreads) extend_tables_kernel(const TableArgs a) {
    // per row of the pass: pages and tokens before it, old length, served
    __shared__ uint32_t s_page[kTableRows + 1], s_tok[kTableRows + 1];
    __shared__ int32_t s_old[kTableRows];
    __shared__ bool s_ok[kTableRows];
    __shared__ uint32_t s_warp[2][kTableThreads / 32];
    // No launch_dependents(): attention reads the page table before it waits for
    // the kernel in front of it, so no later kernel may start before the rows are
    // written.
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ctas = gridDim.x, rank = blockIdx.x;   // the grid is one cluster
    const int P = a.page_size;
    const int shift = 31 - __clz(P);                 // P is a power of two
    const int64_t row_tokens = static_cast<int64_t>(a.max_pages) * P;
    const int32_t num_free = min(max(*a.num_free, 0), a.free_capacity);

    const bool wide = reinterpret_cast<uintptr_t>(a.slot_map) % 16 == 0;
    auto pages_of = [&](int32_t len) { return (static_cast<uint32_t>(len) + P - 1) >> shift; };
    // the free stack's entry for the i-th page of the call
    auto stack_entry = [&](uint32_t i) {
        return a.free_pages + (num_free - 1 - static_cast<int32_t>(i));
    };

    uint32_t pages0 = 0, toks0 = 0;   // before the pass's first row
    uint32_t taken = 0;               // pages of the rows served so far
    for (int r0 = 0; r0 < a.batch; r0 += kTableRows) {
        const int rows = min(kTableRows, a.batch - r0);
        int32_t o = -1, n = 0;
        if (tid < rows) {
            o = a.old_lens[r0 + tid];
            n = a.new_lens[r0 + tid];
        }
        const bool grows = o >= 0 && n >= o;
        const bool fine = grows && n <= row_tokens;
        const uint32_t need = fine ? pages_of(n) - pages_of(o) : 0u;
        uint32_t np = need, nt = grows ? n - o : 0u;   // inclusive sums
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, np, off);
            const uint32_t y = __shfl_up_sync(0xffffffffu, nt, off);
            if (lane >= off) {
                np = sat_add(np, x);
                nt = sat_add(nt, y);
            }
        }
        __syncthreads();   // (the pass before has been read)
        if (lane == 31) {
            s_warp[0][warp] = np;
            s_warp[1][warp] = nt;
        }
        __syncthreads();
        uint32_t pages1 = pages0, toks1 = toks0;   // after the pass's last row
#pragma unroll
        for (int w = 0; w < kTableThreads / 32; ++w) {
            if (w == warp) {
                np = sat_add(np, pages1);
                nt = sat_add(nt, toks1);
            }
            pages1 = sat_add(pages1, s_warp[0][w]);
            toks1 = sat_add(toks1, s_warp[1][w]);
        }
        const bool ok = fine && (need == 0 || np <= static_cast<uint32_t>(num_free));
        if (tid < rows) {
            s_page[tid + 1] = np;
            s_tok[tid + 1] = nt;
            s_old[tid] = o;
            s_ok[tid] = ok;
            if ((r0 + tid) % ctas == rank) {
                a.failed[r0 + tid] = !ok;
                a.cu_tokens[r0 + tid + 1] = static_cast<int32_t>(nt);
            }
        }
        if (tid == 0) {
            s_page[0] = pages0;
            s_tok[0] = toks0;
        }
        __syncthreads();

        // The pass's new table entries: pages [pages0, the last sum that fits).
        if (pages0 <= static_cast<uint32_t>(num_free))
            taken = s_page[last_at_most(s_page, rows + 1, num_free)];
        for (uint32_t i = pages0 + rank * kTableThreads + tid; i < taken; i += ctas * kTableThreads) {
            const int r = last_at_most(s_page, rows, i);
            const int64_t at = static_cast<int64_t>(r0 + r) * a.max_pages + pages_of(s_old[r]) +
                               (i - s_page[r]);
            const int32_t page = *stack_entry(i);
            a.page_table[at] = page;
            if (a.page_tags != nullptr && page >= 0 && page < a.num_pages)
                a.expected_tags[at] = a.page_tags[page];
        }

        // The pass's tokens, kTableTokens consecutive ones at a time: their rows and
        // positions, then all their pages' loads, then the slots.  (Threads counted
        // from the end: a small call's pages and tokens are then different warps.)
        const uint32_t end = min(toks1, static_cast<uint32_t>(a.max_tokens));
        for (uint32_t g = toks0 / kTableTokens + rank * kTableThreads + (kTableThreads - 1 - tid);
             g * kTableTokens < end; g += ctas * kTableThreads) {
            const uint32_t t0 = max(g * kTableTokens, toks0), t1 = min((g + 1) * kTableTokens, end);
            if (t0 >= t1) break;
            const int32_t* from[kTableTokens];   // where a token's page id stands (null: no page)
            int32_t page[kTableTokens], pos[kTableTokens];
            int r = last_at_most(s_tok, rows, t0);
#pragma unroll
            for (int k = 0; k < kTableTokens; ++k) {
                const uint32_t t = g * kTableTokens + k;
                from[k] = nullptr;
                if (t < t0 || t >= t1) continue;
                while (t >= s_tok[r + 1]) ++r;
                if (!s_ok[r]) continue;
                const int32_t old = s_old[r];
                pos[k] = old + static_cast<int32_t>(t - s_tok[r]);
                const int j = pos[k] >> shift, first = pages_of(old);
                from[k] = j >= first ? stack_entry(s_page[r] + (j - first))
                                     : a.page_table + static_cast<int64_t>(r0 + r) * a.max_pages + j;
            }
#pragma unroll
            for (int k = 0; k < kTableTokens; ++k) page[k] = from[k] != nullptr ? *from[k] : -1;
            int32_t slot[kTableTokens];
#pragma unroll
            for (int k = 0; k < kTableTokens; ++k)
                slot[k] = page[k] >= 0 && page[k] < a.num_pages ? page[k] * P + (pos[k] & (P - 1)) : -1;
            if (wide && t1 - t0 == kTableTokens) {
                *reinterpret_cast<int4*>(a.slot_map + t0) =
                    make_int4(slot[0], slot[1], slot[2], slot[3]);
            } else {
#pragma unroll
                for (int k = 0; k < kTableTokens; ++k) {
                    const uint32_t t = g * kTableTokens + k;
                    if (t >= t0 && t < t1) a.slot_map[t] = slot[k];
                }
            }
        }
        pages0 = pages1;
        toks0 = toks1;
    }
    // rows of the slot map behind the last token
    for (int64_t t = static_cast<int64_t>(toks0) + rank * kTableThreads + tid; t < a.max_tokens;
         t += ctas * kTableThreads)
        a.slot_map[t] = -1;
    __threadfence();      // (a kernel that starts on this one's end sees the rows)
    cluster_sync_all();   // every CTA has read num_free
    if (rank == 0 && tid == 0) {
        a.cu_tokens[0] = 0;
        *a.num_free_out = num_free - static_cast<int32_t>(taken);
    }
}

// CTAs: a thread per group of tokens and per row, within one portable cluster.
cudaError_t launch_extend_tables(const TableArgs& a, cudaStream_t stream) {
    const int64_t threads = static_cast<int64_t>(a.max_tokens) / kTableTokens + a.batch;
    int ctas = 1;
    while (ctas < kTableMaxCluster && ctas * kTableThreads < threads) ctas *= 2;
    PdlLaunch l(dim3(ctas), dim3(kTableThreads), 0, stream);
    l.set_cluster(ctas);
    return cudaLaunchKernelEx(&l.cfg, extend_tables_kernel, a);
}

}  // namespace pkv
