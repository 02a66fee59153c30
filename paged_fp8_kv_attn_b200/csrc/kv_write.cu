// kv_write.cu -- the batched page-tag check, the FP8 / BF16 / INT4 append of
// the new token, and the BF16 -> FP8 and BF16 -> INT4 page handoffs.
//
// Source pages: "大模型推理优化：量化、压缩与安全验证", sections "量化 KV cache"
// (FP8 e4m3 cache) and "保护共享 KV cache" (per-page tags, per-request
// expected tags, check before a decode op reads the cache, abort on
// mismatch, done as a separate batched check); siami.tw editorial, section
// "共享 KV 快取的完整性檢查" (Table 3 and the note that the check is not fused
// into the attention kernel).
#include "device.cuh"
#include "internal.h"
#include "kv_codec.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// tag check: one CTA per request; threads stride over its used entries
// ---------------------------------------------------------------------------
constexpr int kTagThreads = 128;

__global__ void __launch_bounds__(kTagThreads)
tag_check_kernel(const uint32_t* __restrict__ page_tags, int32_t num_pages,
                 const int32_t* __restrict__ page_table,
                 const uint32_t* __restrict__ expected_tags, int32_t max_pages,
                 const int32_t* __restrict__ seq_lens, int32_t page_size, int32_t window,
                 int32_t sinks, uint8_t* __restrict__ abort_out,
                 int32_t* __restrict__ num_aborted) {
    // Let the next kernel on the stream launch at once (its own prologue
    // overlaps this grid); it still waits for this grid to finish before it
    // reads anything this grid writes.
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x;
    const int32_t L = seq_lens[b];
    int bad = (L < 1 || static_cast<int64_t>(L) > static_cast<int64_t>(max_pages) * page_size);
    if (!bad) {
        // (window > 0: entries [skip, skip + gap) hold hidden tokens only)
        int32_t used = blocks_of(L, page_size), skip = used, gap = 0;
        if (window > 0) {
            const int32_t lo = L > window ? L - window : 0;
            const int32_t s = sinks < lo ? sinks : lo;
            skip = s > 0 ? blocks_of(s, page_size) : 0;
            gap = lo / page_size > skip ? lo / page_size - skip : 0;
            used -= gap;
        }
        const int32_t* row = page_table + static_cast<int64_t>(b) * max_pages;
        const uint32_t* exp = expected_tags + static_cast<int64_t>(b) * max_pages;
#pragma unroll 4
        for (int i = threadIdx.x; i < used; i += kTagThreads) {
            const int j = i < skip ? i : i + gap;
            const int32_t pid = row[j];
            const uint32_t want = exp[j];
            if (pid < 0 || pid >= num_pages)
                bad = 1;
            else if (__ldg(page_tags + pid) != want)
                bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        abort_out[b] = static_cast<uint8_t>(bad != 0);
        if (bad && num_aborted) atomicAdd(num_aborted, 1);
    }
}

cudaError_t launch_tag_check(const uint32_t* page_tags, int32_t num_pages,
                             const int32_t* page_table, const uint32_t* expected_tags,
                             int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                             int32_t page_size, int32_t window, int32_t sinks, uint8_t* abort_out,
                             int32_t* num_aborted, cudaStream_t stream) {
    PdlLaunch l(dim3(batch), dim3(kTagThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, tag_check_kernel, page_tags, num_pages, page_table,
                              expected_tags, max_pages, seq_lens, page_size, window, sinks,
                              abort_out, num_aborted);
}

// ---------------------------------------------------------------------------
// append: one CTA per request
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

template <int kKv>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
              const int32_t* __restrict__ page_table, int32_t max_pages,
              const int32_t* __restrict__ seq_lens, int32_t num_kv_heads, int32_t head_dim,
              int32_t page_size, float k_scale, float v_scale, void* __restrict__ k_cache,
              void* __restrict__ v_cache, uint32_t* __restrict__ k_params,
              uint32_t* __restrict__ v_params, int32_t num_pages,
              const uint8_t* __restrict__ abort) {
    // Let the next kernel on the stream launch at once (its own prologue
    // overlaps this grid); it still waits for this grid to finish before it
    // reads anything this grid writes.
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x;
    const int32_t L = seq_lens[b];
    if (L < 1 || static_cast<int64_t>(L) > static_cast<int64_t>(max_pages) * page_size) return;
    if (abort != nullptr && abort[b] != 0) return;
    const int32_t pos = L - 1;
    const int32_t pid = page_table[static_cast<int64_t>(b) * max_pages + pos / page_size];
    if (pid < 0 || pid >= num_pages) return;
    const int32_t slot = pos % page_size;
    const int per_tensor = num_kv_heads * (head_dim / 8);
    for (int e = threadIdx.x; e < 2 * per_tensor; e += kAppendThreads) {
        const bool is_v = e >= per_tensor;
        const int r = is_v ? e - per_tensor : e;
        const int h = r / (head_dim / 8);
        const int d8 = r % (head_dim / 8);
        const uint16_t* src = (is_v ? v_new : k_new) +
                              (static_cast<int64_t>(b) * num_kv_heads + h) * head_dim + d8 * 8;
        const uint4 raw = *reinterpret_cast<const uint4*>(src);
        const int64_t dst = (static_cast<int64_t>(pid) * num_kv_heads + h) * page_size + slot;
        store8<kKv>(is_v ? v_cache : k_cache, is_v ? v_params : k_params, dst, head_dim, d8, raw,
                    is_v ? v_scale : k_scale);
    }
}

cudaError_t launch_append(const KvDst& dst, const uint16_t* k_new, const uint16_t* v_new,
                          const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                          int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                          int32_t page_size, int32_t num_pages, const uint8_t* abort,
                          cudaStream_t stream) {
    PdlLaunch l(dim3(batch), dim3(kAppendThreads), 0, stream);
    auto* kernel = dst.kv == kKvFp8    ? append_kernel<kKvFp8>
                   : dst.kv == kKvBf16 ? append_kernel<kKvBf16>
                                       : append_kernel<kKvInt4>;
    return cudaLaunchKernelEx(&l.cfg, kernel, k_new, v_new, page_table, max_pages, seq_lens,
                              num_kv_heads, head_dim, page_size, dst.k_scale, dst.v_scale, dst.k,
                              dst.v, dst.k_params, dst.v_params, num_pages, abort);
}

// ---------------------------------------------------------------------------
// fused check + append: one CTA per request.  The request's tag check and its
// append depend on nothing but the request itself, so one CTA checks the used
// entries while the new token's K/V are already being loaded, and writes the
// token only if the request passed.  Results are those of kv_tag_check
// followed by kv_append_* with its abort mask.
// ---------------------------------------------------------------------------
constexpr int kFusedThreads = 256;

template <int kKv>
__global__ void __launch_bounds__(kFusedThreads)
check_append_kernel(const uint32_t* __restrict__ page_tags, int32_t num_pages,
                    const int32_t* __restrict__ page_table,
                    const uint32_t* __restrict__ expected_tags, int32_t max_pages,
                    const int32_t* __restrict__ seq_lens, int32_t page_size,
                    const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
                    int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                    void* __restrict__ k_cache, void* __restrict__ v_cache,
                    uint32_t* __restrict__ k_params, uint32_t* __restrict__ v_params,
                    uint8_t* __restrict__ abort_out, int32_t* __restrict__ num_aborted) {
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x;
    const int per_tensor = num_kv_heads * (head_dim / 8);
    const int32_t* row = page_table + static_cast<int64_t>(b) * max_pages;
    const uint32_t* exp = expected_tags + static_cast<int64_t>(b) * max_pages;
    // One round trip for everything that does not depend on the length: the
    // length itself, this thread's first page-table entry and expected tag,
    // and the new token's values for this thread's first two 8-element groups.
    const int32_t L = seq_lens[b];
    const int j0 = threadIdx.x;
    const int32_t p_first = j0 < max_pages ? row[j0] : -1;
    const uint32_t e_first = j0 < max_pages ? exp[j0] : 0u;
    uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int e = threadIdx.x + k * kFusedThreads;
        if (e < 2 * per_tensor) {
            const bool is_v = e >= per_tensor;
            const int r = is_v ? e - per_tensor : e;
            const int h = r / (head_dim / 8), d8 = r % (head_dim / 8);
            raw[k] = *reinterpret_cast<const uint4*>(
                (is_v ? v_new : k_new) + (static_cast<int64_t>(b) * num_kv_heads + h) * head_dim +
                d8 * 8);
        }
    }
    int bad = (L < 1 || static_cast<int64_t>(L) > static_cast<int64_t>(max_pages) * page_size);
    int32_t pid = -1, slot = 0;
    if (!bad) {
        const int32_t pos = L - 1;
        slot = pos % page_size;
        const int32_t used = blocks_of(L, page_size);
        pid = row[pos / page_size];
        for (int j = j0; j < used; j += kFusedThreads) {
            const int32_t p = (j == j0) ? p_first : row[j];
            const uint32_t want = (j == j0) ? e_first : exp[j];
            if (p < 0 || p >= num_pages)
                bad = 1;
            else if (__ldg(page_tags + p) != want)
                bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        abort_out[b] = static_cast<uint8_t>(bad != 0);
        if (bad && num_aborted) atomicAdd(num_aborted, 1);
    }
    if (bad) return;   // an aborted request writes nothing (its last page id was checked too)
    int k = 0;
    for (int e = threadIdx.x; e < 2 * per_tensor; e += kFusedThreads, ++k) {
        const bool is_v = e >= per_tensor;
        const int r = is_v ? e - per_tensor : e;
        const int h = r / (head_dim / 8), d8 = r % (head_dim / 8);
        uint4 val;
        if (k == 0)
            val = raw[0];
        else if (k == 1)
            val = raw[1];
        else
            val = *reinterpret_cast<const uint4*>(
                (is_v ? v_new : k_new) + (static_cast<int64_t>(b) * num_kv_heads + h) * head_dim +
                d8 * 8);
        const int64_t dst = (static_cast<int64_t>(pid) * num_kv_heads + h) * page_size + slot;
        store8<kKv>(is_v ? v_cache : k_cache, is_v ? v_params : k_params, dst, head_dim, d8, val,
                    is_v ? v_scale : k_scale);
    }
}

cudaError_t launch_check_append(const KvDst& dst, const uint32_t* page_tags, int32_t num_pages,
                                const int32_t* page_table, const uint32_t* expected_tags,
                                int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                int32_t page_size, const uint16_t* k_new, const uint16_t* v_new,
                                int32_t num_kv_heads, int32_t head_dim, uint8_t* abort_out,
                                int32_t* num_aborted, cudaStream_t stream) {
    PdlLaunch l(dim3(batch), dim3(kFusedThreads), 0, stream);
    auto* kernel = dst.kv == kKvFp8    ? check_append_kernel<kKvFp8>
                   : dst.kv == kKvBf16 ? check_append_kernel<kKvBf16>
                                       : check_append_kernel<kKvInt4>;
    return cudaLaunchKernelEx(&l.cfg, kernel, page_tags, num_pages, page_table, expected_tags,
                              max_pages, seq_lens, page_size, k_new, v_new, num_kv_heads, head_dim,
                              dst.k_scale, dst.v_scale, dst.k, dst.v, dst.k_params, dst.v_params,
                              abort_out, num_aborted);
}

// ---------------------------------------------------------------------------
// page reallocation bookkeeping: tag bumps and expected-tag rebuilds
// ("保护共享 KV cache": a page's tag changes whenever it is reallocated; the
// server records each request's expected tags)
// ---------------------------------------------------------------------------
constexpr int kTagOpThreads = 256;

__global__ void __launch_bounds__(kTagOpThreads)
retag_kernel(uint32_t* __restrict__ page_tags, int32_t num_pages,
             const int32_t* __restrict__ pages, int32_t n) {
    launch_dependents();
    grid_dependency_wait();
    for (int i = blockIdx.x * kTagOpThreads + threadIdx.x; i < n; i += gridDim.x * kTagOpThreads) {
        const int32_t p = pages[i];
        if (p >= 0 && p < num_pages) atomicAdd(page_tags + p, 1u);   // wraps mod 2^32
    }
}

__global__ void __launch_bounds__(kTagOpThreads)
expected_tags_kernel(const uint32_t* __restrict__ page_tags, int32_t num_pages,
                     const int32_t* __restrict__ page_table, int32_t max_pages,
                     const int32_t* __restrict__ seq_lens, int32_t page_size,
                     uint32_t* __restrict__ expected_tags) {
    launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x;
    const int32_t L = seq_lens[b];
    if (L < 1 || static_cast<int64_t>(L) > static_cast<int64_t>(max_pages) * page_size) return;
    const int32_t used = blocks_of(L, page_size);
    const int64_t row = static_cast<int64_t>(b) * max_pages;
    for (int j = threadIdx.x; j < used; j += kTagOpThreads) {
        const int32_t p = page_table[row + j];
        if (p >= 0 && p < num_pages) expected_tags[row + j] = page_tags[p];
    }
}

cudaError_t launch_retag(uint32_t* page_tags, int32_t num_pages, const int32_t* pages, int32_t n,
                         cudaStream_t stream) {
    int blocks = (n + kTagOpThreads - 1) / kTagOpThreads;
    if (blocks > 1024) blocks = 1024;
    PdlLaunch l(dim3(blocks), dim3(kTagOpThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, retag_kernel, page_tags, num_pages, pages, n);
}

cudaError_t launch_expected_tags(const uint32_t* page_tags, int32_t num_pages,
                                 const int32_t* page_table, int32_t max_pages,
                                 const int32_t* seq_lens, int32_t batch, int32_t page_size,
                                 uint32_t* expected_tags, cudaStream_t stream) {
    PdlLaunch l(dim3(batch), dim3(kTagOpThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, expected_tags_kernel, page_tags, num_pages, page_table,
                              max_pages, seq_lens, page_size, expected_tags);
}

// ---------------------------------------------------------------------------
// BF16 -> FP8 (INT4) page handoff: grid-stride over 16-element groups (8-element
// blocks)
// ---------------------------------------------------------------------------
constexpr int kRequantThreads = 256;

__global__ void __launch_bounds__(kRequantThreads)
requant_kernel(const uint16_t* __restrict__ src_pool, int32_t src_num_pages,
               const int32_t* __restrict__ src_pages, uint8_t* __restrict__ dst_pool,
               int32_t dst_num_pages, const int32_t* __restrict__ dst_pages, int32_t num_pairs,
               int64_t page_elems, float scale) {
    // Let the next kernel on the stream launch at once (its own prologue
    // overlaps this grid); it still waits for this grid to finish before it
    // reads anything this grid writes.
    launch_dependents();
    grid_dependency_wait();
    const int64_t groups = page_elems / 16;
    const int64_t total = static_cast<int64_t>(num_pairs) * groups;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int32_t pair = static_cast<int32_t>(i / groups);
        const int64_t gi = i % groups;
        const int32_t s = src_pages[pair];
        const int32_t d = dst_pages[pair];
        if (s < 0 || s >= src_num_pages || d < 0 || d >= dst_num_pages) continue;
        const uint4* sp = reinterpret_cast<const uint4*>(src_pool + s * page_elems + gi * 16);
        const uint2 lo = quantize8(sp[0], scale);
        const uint2 hi = quantize8(sp[1], scale);
        *reinterpret_cast<uint4*>(dst_pool + d * page_elems + gi * 16) =
            make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

// INT4: 8 values a thread, a group of 64 in 8 consecutive lanes (page_elems is
// a multiple of 64, so a group never spans two pairs or the end).
__global__ void __launch_bounds__(kRequantThreads)
requant_int4_kernel(const uint16_t* __restrict__ src_pool, int32_t src_num_pages,
                    const int32_t* __restrict__ src_pages, uint8_t* __restrict__ dst_codes,
                    uint32_t* __restrict__ dst_params, int32_t dst_num_pages,
                    const int32_t* __restrict__ dst_pages, int32_t num_pairs, int64_t page_elems,
                    int32_t head_dim) {
    launch_dependents();
    grid_dependency_wait();
    const int64_t blocks = page_elems / 8;
    const int64_t total = static_cast<int64_t>(num_pairs) * blocks;
    const int per_row = head_dim / 8;
    for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int32_t pair = static_cast<int32_t>(i / blocks);
        const int64_t bi = i % blocks;
        const int32_t s = src_pages[pair];
        const int32_t d = dst_pages[pair];
        if (s < 0 || s >= src_num_pages || d < 0 || d >= dst_num_pages) continue;
        const uint4 raw = *reinterpret_cast<const uint4*>(src_pool + s * page_elems + bi * 8);
        store8<kKvInt4>(dst_codes, dst_params, (d * page_elems) / head_dim + bi / per_row, head_dim,
                        static_cast<int>(bi % per_row), raw, 1.f);
    }
}

static int64_t requant_blocks(int64_t threads) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t blocks = (threads + kRequantThreads - 1) / kRequantThreads;
    const int64_t cap = static_cast<int64_t>(sms) * 8;
    return blocks > cap ? cap : (blocks < 1 ? 1 : blocks);
}

cudaError_t launch_requant_int4(const uint16_t* src_pool, int32_t src_num_pages,
                                const int32_t* src_pages, uint8_t* dst_codes,
                                uint32_t* dst_params, int32_t dst_num_pages,
                                const int32_t* dst_pages, int32_t num_pairs, int64_t page_elems,
                                int32_t head_dim, cudaStream_t stream) {
    const int64_t blocks = requant_blocks(static_cast<int64_t>(num_pairs) * (page_elems / 8));
    PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(kRequantThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, requant_int4_kernel, src_pool, src_num_pages, src_pages,
                              dst_codes, dst_params, dst_num_pages, dst_pages, num_pairs,
                              page_elems, head_dim);
}

cudaError_t launch_requant(const uint16_t* src_pool, int32_t src_num_pages,
                           const int32_t* src_pages, uint8_t* dst_pool, int32_t dst_num_pages,
                           const int32_t* dst_pages, int32_t num_pairs, int64_t page_elems,
                           float scale, cudaStream_t stream) {
    const int64_t blocks = requant_blocks(static_cast<int64_t>(num_pairs) * (page_elems / 16));
    PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(kRequantThreads), 0, stream);
    return cudaLaunchKernelEx(&l.cfg, requant_kernel, src_pool, src_num_pages, src_pages,
                              dst_pool, dst_num_pages, dst_pages, num_pairs, page_elems, scale);
}

// The step's first kernels run beside the attention grid that programmatic
// dependent launch starts early: an SM running one of them must already have
// its on-chip memory configured as the attention kernel wants it (all of it
// shared), or the attention CTAs can join that SM only after it drains.
cudaError_t step_kernels_set_carveout() {
    const int c = cudaSharedmemCarveoutMaxShared;
    const cudaFuncAttribute at = cudaFuncAttributePreferredSharedMemoryCarveout;
    cudaError_t e = cudaFuncSetAttribute(tag_check_kernel, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(append_kernel<kKvFp8>, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(append_kernel<kKvBf16>, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(append_kernel<kKvInt4>, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(check_append_kernel<kKvFp8>, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(check_append_kernel<kKvBf16>, at, c);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(check_append_kernel<kKvInt4>, at, c);
    return e;
}

}  // namespace pkv
