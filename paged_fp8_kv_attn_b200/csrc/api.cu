// api.cu -- the extern "C" entry points declared in include/pagedkv.h:
// host-side argument validation, TMA descriptor encoding, workspace layout
// and kernel launches.  No call allocates, frees or synchronises.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "internal.h"
#include "pagedkv.h"

namespace {

thread_local std::string g_last_error;

pkv_status fail(pkv_status code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return code;
}

pkv_status cuda_fail(cudaError_t e, const char* what) {
    return fail(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

bool known_kv(int32_t kv) {
    return kv == PKV_KV_FP8 || kv == PKV_KV_BF16 || kv == PKV_KV_INT4;
}
bool supported_head_dim(int32_t d) { return d == 64 || d == 128; }
bool supported_page_size(int32_t p) { return p == 16 || p == 32 || p == 64 || p == 128; }

// ---------------------------------------------------------------------------
// per-device launch limits (SM count, resident attention CTAs per SM)
// ---------------------------------------------------------------------------
constexpr int kMaxDevices = 64;
struct DeviceInfo {
    bool ready = false;
    int sms = 0;
    // [cache type][d128][gp16][two KV heads per item][window]
    int occupancy[3][2][2][2][2] = {};
    // resident clusters of each size (index = cluster size; -1 = not queried);
    // read without the lock
    mutable std::atomic<int> clusters[3][2][2][2][2][pkv::kMaxCluster + 1];
};
std::mutex g_dev_mutex;
DeviceInfo g_dev[kMaxDevices];

pkv_status device_info(const DeviceInfo** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(PKV_ERR_UNSUPPORTED, "device index %d", dev);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    DeviceInfo& info = g_dev[dev];
    if (!info.ready) {
        e = cudaDeviceGetAttribute(&info.sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
        e = pkv::step_kernels_set_carveout();
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        for (int i = 0; i < 3 * 16; ++i) {
            const int kv = i / 16, d = i & 1, gp = (i >> 1) & 1, h2 = (i >> 2) & 1, w = (i >> 3) & 1;
            const pkv::AttnVariant v{kv, d ? 128 : 64, gp ? 16 : 8, h2 ? 2 : 1, w == 1};
            if (pkv::attn_partial_smem_bytes(v) == 0) continue;
            e = pkv::attn_set_smem_attr(v);
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
            int blocks = 0;
            e = pkv::attn_occupancy(v, &blocks);
            if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
            info.occupancy[kv][d][gp][h2][w] = blocks < 1 ? 1 : blocks;
            for (int c = 0; c <= pkv::kMaxCluster; ++c) info.clusters[kv][d][gp][h2][w][c] = -1;
        }
        info.ready = true;
    }
    *out = &info;
    return PKV_OK;
}

int group_pad_of(int group) { return group <= 8 ? 8 : 16; }

pkv::AttnVariant variant_of(int kv, int head_dim, int group, int kv_per_item, bool window) {
    return {kv, head_dim, group_pad_of(group), kv_per_item, window};
}

// Clusters of `size` CTAs of this attention variant that fit on the device at
// once (queried once per device, variant and size).
int max_clusters(const DeviceInfo& info, const pkv::AttnVariant& v, int size) {
    std::atomic<int>& slot =
        info.clusters[v.kv][v.head_dim == 128][v.group_pad == 16][v.kv_per_item == 2][v.window][size];
    if (slot < 0) {
        std::lock_guard<std::mutex> lock(g_dev_mutex);
        int n = 0;
        cudaError_t e = pkv::attn_max_clusters(v, size, &n);
        if (e != cudaSuccess) {
            cudaGetLastError();   // a refused shape is an answer, not a sticky error
            n = 0;
        }
        slot = n;
    }
    return slot;
}

// Cluster mode for `items` work items: cluster size C and K clusters, each
// owning ceil(items / K) or fewer whole items.  With `forced` > 0 the size is
// given; otherwise the size maximising C * items / (items per cluster) -- the
// CTAs kept busy, discounted by the imbalance of whole items per cluster --
// over 2..kMaxCluster.  Among sizes that tie, the largest portable one (at
// most 8) wins: more CTAs share each cluster's items, which evens out
// requests of unequal length.  Returns C = 0 when no cluster shape fits.
pkv_status choose_clusters(const pkv::AttnVariant& v, int64_t items, int forced, int* size,
                           int* count) {
    *size = 0;
    *count = 0;
    const DeviceInfo* info = nullptr;
    pkv_status st = device_info(&info);
    if (st != PKV_OK) return st;
    double best = 0.0;
    const int c_lo = forced > 0 ? forced : 2;
    const int c_hi = forced > 0 ? forced : pkv::kMaxCluster;
    for (int c = c_lo; c <= c_hi; ++c) {
        const int kmax = max_clusters(*info, v, c);
        if (kmax <= 0) continue;
        const int64_t k = std::min<int64_t>(items, kmax);
        const int64_t per = (items + k - 1) / k;            // items of the fullest cluster
        const double score = static_cast<double>(c) * static_cast<double>(items) / per;
        if (score > best || (score == best && c <= 8)) {
            best = score;
            *size = c;
            *count = static_cast<int>((items + per - 1) / per);
        }
    }
    return PKV_OK;
}

pkv_status default_ctas(const pkv::AttnVariant& v, int* ctas) {
    const DeviceInfo* info = nullptr;
    pkv_status st = device_info(&info);
    if (st != PKV_OK) return st;
    *ctas = info->sms * info->occupancy[v.kv][v.head_dim == 128][v.group_pad == 16]
                                       [v.kv_per_item == 2][v.window];
    return PKV_OK;
}

// ---------------------------------------------------------------------------
// TMA descriptors for the K / V pools viewed as 2-D [rows][head_dim]
// ---------------------------------------------------------------------------
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

pkv_status get_encoder(EncodeTiledFn* fn) {
    static std::once_flag once;
    static EncodeTiledFn cached = nullptr;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        err = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
        if (err == cudaSuccess && q == cudaDriverEntryPointSuccess)
            cached = reinterpret_cast<EncodeTiledFn>(p);
    });
    if (cached == nullptr)
        return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(err));
    *fn = cached;
    return PKV_OK;
}

pkv_status encode_pool_map(CUtensorMap* map, const void* pool, int kv, int head_dim,
                           int64_t rows, int box_rows) {
    EncodeTiledFn encode = nullptr;
    pkv_status st = get_encoder(&encode);
    if (st != PKV_OK) return st;
    const bool bytes = kv != PKV_KV_BF16;
    // row elements: codes (FP8), pairs of codes (INT4) or bf16 values
    const int inner = kv == PKV_KV_INT4 ? head_dim / 2 : head_dim;
    const int esize = bytes ? 1 : 2;
    const int box_inner = bytes ? inner : 64;   // elements; 32, 64 or 128 bytes
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner) * esize};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapSwizzle sw = (box_inner * esize == 128)  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : (box_inner * esize == 64) ? CU_TENSOR_MAP_SWIZZLE_64B
                                                              : CU_TENSOR_MAP_SWIZZLE_NONE;
    CUresult r = encode(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                        2, const_cast<void*>(pool), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return PKV_OK;
}

// Generic 2-D map: `rows` rows of `inner` elements, rows `row_bytes` apart.
pkv_status encode_2d(CUtensorMap* map, CUtensorMapDataType dtype, const void* base,
                     uint64_t inner, uint64_t rows, uint64_t row_bytes, uint32_t box_inner,
                     uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    EncodeTiledFn encode = nullptr;
    pkv_status st = get_encoder(&encode);
    if (st != PKV_OK) return st;
    cuuint64_t dims[2] = {inner, rows};
    cuuint64_t strides[1] = {row_bytes};
    cuuint32_t box[2] = {box_inner, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = encode(map, dtype, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(PKV_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return PKV_OK;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

pkv_status check_common_kv(int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                           int32_t page_size, int32_t num_pages, int32_t max_pages) {
    if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch must be >= 0 (got %d)", batch);
    if (num_kv_heads < 1) return fail(PKV_ERR_INVALID_ARG, "num_kv_heads must be >= 1");
    if (!supported_head_dim(head_dim))
        return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", head_dim);
    if (!supported_page_size(page_size))
        return fail(PKV_ERR_UNSUPPORTED, "page_size %d not supported (16, 32, 64, 128)", page_size);
    if (num_pages < 1) return fail(PKV_ERR_INVALID_ARG, "num_pages must be >= 1");
    if (max_pages < 1) return fail(PKV_ERR_INVALID_ARG, "max_pages must be >= 1");
    const int64_t rows = static_cast<int64_t>(num_pages) * num_kv_heads * page_size;
    if (rows >= (int64_t(1) << 31))
        return fail(PKV_ERR_UNSUPPORTED, "num_pages * num_kv_heads * page_size must be < 2^31");
    return PKV_OK;
}

// The attention kernels count a batch's 64-token chunks in 32 bits.
pkv_status check_chunks(int32_t batch, int32_t max_pages, int32_t page_size) {
    const int64_t chunks = (static_cast<int64_t>(max_pages) * page_size - 1) / pkv::kChunkTokens + 1;
    if (chunks * batch > INT32_MAX)
        return fail(PKV_ERR_UNSUPPORTED, "batch * ceil(max_pages * page_size / 64) must be < 2^31");
    return PKV_OK;
}

// The work split of one attention call (see paged_decode_attn_plan).
struct AttnPlan {
    int kv_per_item;      // KV heads per work item the kernel uses
    int ws_kv_per_item;   // the one the workspace is sized for
    int grid;             // split-K grid (also sizes the workspace)
    int cluster;          // 0: split-K + merge; C > 0: clusters of C CTAs
    int nclusters;
};

// The most tokens a request can attend to (window > 0: with that window).
int64_t max_visible(int32_t max_pages, int32_t page_size, int32_t window, int32_t sinks) {
    const int64_t all = static_cast<int64_t>(max_pages) * page_size;
    return window > 0 ? std::min<int64_t>(all, static_cast<int64_t>(window) + sinks) : all;
}

// Whether the library's work split of a call comes from model_split (INT4 caches
// and windows) or from plan_attention's rule on the item count (FP8 and BF16
// without a window).
bool modelled_split(int kv, int32_t window) { return kv == PKV_KV_INT4 || window > 0; }

// Work split from an estimate of the slowest CTA's time, in us, at the longest
// requests that the page table allows: a chunk costs more the more CTAs share an
// SM, a segment (an item's part in a CTA: its prologue and epilogue) about as much
// as two chunks, clusters of several CTAs their two barriers, split-K its merge
// launch.  Constants from a B200: one chunk of a lone CTA 0.9 (INT4, two heads of
// 128), 0.77 (FP8 two heads, BF16 one); 1.7 at three and 1.4 at two CTAs per SM;
// items of one head 0.65 of two, heads of 64 dims 0.65 of 128; and no less than
// 0.07 for each TMA box of a chunk, which one lane issues.
// Requests of one batch differ in length, which split-K evens out and whole items
// do not: a cluster's chunks count 25% more, but for a window shorter than the
// table's longest request, which makes most of them equal (96 requests of up to
// 8,190 tokens, 64 dims: clusters of one 114, split-K 79; that one batch set the 25%).
// Measured cold, this choice / the item-count rule: INT4 64 x 8,192 tokens 137 / 150
// (split-K), 2 x 131,072 82 / 128 (split-K), 128 x 16 22 / 32 (clusters of one; with
// a table much wider than the requests split-K, 25), FP8 window of 400 over 128 x 600
// 37 / 48 (clusters of one), INT4 window of 16,384 over 8 x 65,536 58 / 57 (split-K).
pkv_status model_split(int kv, int head_dim, int group, bool window, int page_size, int32_t batch,
                       int64_t items, int wide, int64_t chunks, int grid, int* kv_per_item,
                       int* cluster, int* nclusters) {
    const DeviceInfo* info = nullptr;
    pkv_status st = device_info(&info);
    if (st != PKV_OK) return st;
    constexpr double kSegment = 3.0, kBarriers = 3.0, kMerge = 6.0;
    const double uneven = window ? 1.0 : 1.0 + 0.25 * (1.0 - 1.0 / batch);
    auto chunk = [&](double ctas, int heads) {
        const double shared = std::max(0.0, ctas / info->sms - 1.0);
        const double t = kv == PKV_KV_INT4 ? 0.9 + 0.4 * shared : 0.77 + 0.63 * shared;
        int boxes = 2 * std::max(1, pkv::kChunkTokens / page_size);
        if (kv == PKV_KV_BF16 && head_dim == 128) boxes *= 2;
        if (kv == PKV_KV_INT4) boxes = page_size <= pkv::int4_direct_page(head_dim) ? 0 : 2 * boxes;
        const bool joint = kv == PKV_KV_INT4 ? page_size <= pkv::kChunkTokens
                                             : page_size == pkv::kChunkTokens;
        if (heads == 2 && !joint) boxes *= 2;
        return std::max(t * (heads < 2 && kv != PKV_KV_BF16 ? 0.65 : 1.0) *
                            (head_dim == 64 ? 0.65 : 1.0),
                        0.07 * boxes);
    };
    *kv_per_item = wide;
    *cluster = *nclusters = 0;
    const double n = static_cast<double>(items);
    double best = n * chunks / grid * chunk(grid, wide) + (n / grid + 1.0) * kSegment + kMerge;
    // (few two-head items may be taken one head at a time, which doubles them)
    for (int heads = wide; heads >= 1; --heads) {
        if (heads < wide && items * 4 > info->sms) break;
        const int64_t parts = items * (wide / heads);
        const pkv::AttnVariant v = variant_of(kv, head_dim, group, heads, window);
        for (int c = 1; c <= pkv::kMaxCluster; ++c) {
            const int kmax = max_clusters(*info, v, c);
            if (kmax <= 0) continue;
            const int64_t k = std::min<int64_t>(parts, kmax);
            const int64_t most = (parts + k - 1) / k;   // items of the fullest cluster
            const double per = static_cast<double>(most);
            const double t = uneven * per * chunks / c * chunk(static_cast<double>(k) * c, heads) +
                             (c == 1 ? per * kSegment : (per / c + 1.0) * kSegment + kBarriers);
            if (t < best) {
                best = t;
                *kv_per_item = heads;
                *cluster = c;
                *nclusters = static_cast<int>((parts + most - 1) / most);
            }
        }
    }
    return PKV_OK;
}

pkv_status plan_attention(int kv, int32_t batch, int32_t num_kv_heads, int32_t group,
                          int32_t head_dim, int32_t max_pages, int32_t page_size, int32_t window,
                          int32_t sinks, int32_t num_ctas, AttnPlan* plan,
                          bool allow_cluster = true) {
    pkv_status st = PKV_OK;
    int kv_per_item = pkv::kv_heads_per_item(kv, num_kv_heads, group);
    plan->ws_kv_per_item = kv_per_item;
    int grid = num_ctas > 0 ? num_ctas : 0;
    if (grid == 0) {
        // one wave of resident CTAs, but no more than leaves each CTA about
        // eight 64-token chunks of the largest batch the page table allows
        // (small batches gain from fewer, longer segments and a lighter merge)
        st = default_ctas(variant_of(kv, head_dim, group, kv_per_item, window > 0), &grid);
        if (st != PKV_OK) return st;
        const DeviceInfo* info = nullptr;
        st = device_info(&info);
        if (st != PKV_OK) return st;
        const int64_t chunks_per_seq =
            (max_visible(max_pages, page_size, window, sinks) + pkv::kChunkTokens - 1) /
            pkv::kChunkTokens;
        const int64_t max_units =
            static_cast<int64_t>(batch) * (num_kv_heads / kv_per_item) * chunks_per_seq;
        int64_t cap = std::max<int64_t>(info->sms, (max_units + 7) / 8);
        // INT4 and windows: nor fewer CTAs than items (short requests; measured cold with
        // 128 x 16 tokens, 512 items: 25.0 us on 444 CTAs, 32.0 on 148)
        if (modelled_split(kv, window))
            cap = std::max<int64_t>(cap, static_cast<int64_t>(batch) * (num_kv_heads / kv_per_item));
        if (cap < grid) grid = static_cast<int>(cap);
    } else {
        const DeviceInfo* info = nullptr;
        st = device_info(&info);  // sets the shared-memory attribute
        if (st != PKV_OK) return st;
    }
    plan->grid = grid;
    // Cluster mode (no merge kernel): the library's choice (num_ctas == 0)
    // when the batch has no more items than one wave of CTAs (measured on
    // B200: faster than split-K plus merge at every such size of the
    // concurrency sweep; larger batches, which can be ragged, keep the
    // balanced split-K partition), or requested with num_ctas = -C.  With at
    // most a quarter as many two-head items as SMs (up to 9 requests at 8 KV
    // heads), the library's choice takes one KV head per item, which doubles
    // the items and the CTAs that share them (measured on B200 at 8,192
    // tokens: 13% faster at 4 requests, unchanged at 1 and 8, 4-5% slower at
    // 16 and 32; cluster mode needs the workspace for its status word only,
    // so the workspace size does not depend on this).
    int64_t items = static_cast<int64_t>(batch) * (num_kv_heads / kv_per_item);
    int cluster = 0, nclusters = 0;
    if (allow_cluster && num_ctas == 0 && modelled_split(kv, window)) {
        st = model_split(kv, head_dim, group, window > 0, page_size, batch, items, kv_per_item,
                         (max_visible(max_pages, page_size, window, sinks) + pkv::kChunkTokens - 1) /
                             pkv::kChunkTokens,
                         grid, &kv_per_item, &cluster, &nclusters);
        if (st != PKV_OK) return st;
    } else if (allow_cluster && (num_ctas < 0 || (num_ctas == 0 && items <= grid))) {
        if (num_ctas == 0 && kv_per_item == 2) {
            const DeviceInfo* info = nullptr;
            st = device_info(&info);
            if (st != PKV_OK) return st;
            if (items * 4 <= info->sms) {
                kv_per_item = 1;
                items *= 2;
            }
        }
        st = choose_clusters(variant_of(kv, head_dim, group, kv_per_item, window > 0), items,
                             num_ctas < 0 ? -num_ctas : 0, &cluster, &nclusters);
        if (st != PKV_OK) return st;
        if (cluster == 0 && num_ctas < 0)
            return fail(PKV_ERR_UNSUPPORTED, "clusters of %d CTAs do not fit on this device",
                        -num_ctas);
    }
    plan->kv_per_item = kv_per_item;
    plan->cluster = cluster;
    plan->nclusters = nclusters;
    return PKV_OK;
}

// The K and V pools of one attention call.
struct KvPools {
    int kv;                      // PKV_KV_*
    const void* k;
    const void* v;
    float k_scale, v_scale;      // FP8
    const uint16_t* k_params;    // INT4
    const uint16_t* v_params;
};

// window > 0: only the last `window` and the first `sinks` tokens are visible.
pkv_status attn_impl(const KvPools& pools, const uint16_t* q, const int32_t* page_table,
                     int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                     int32_t page_size, int32_t num_pages, float sm_scale, int32_t window,
                     int32_t sinks, const uint8_t* abort, uint16_t* out, float* lse,
                     void* workspace, size_t workspace_bytes, int32_t num_ctas, void* stream) {
    const int kv = pools.kv;
    const bool fp8 = kv == PKV_KV_FP8, int4 = kv == PKV_KV_INT4;
    const void *k_cache = pools.k, *v_cache = pools.v;
    const float k_scale = pools.k_scale, v_scale = pools.v_scale;
    pkv_status st = check_common_kv(batch, num_kv_heads, head_dim, page_size, num_pages, max_pages);
    if (st != PKV_OK) return st;
    if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(PKV_ERR_INVALID_ARG, "num_q_heads (%d) must be a positive multiple of "
                    "num_kv_heads (%d)", num_q_heads, num_kv_heads);
    const int group = num_q_heads / num_kv_heads;
    if (group > 16) return fail(PKV_ERR_UNSUPPORTED, "GQA group %d > 16 not supported", group);
    if (!(std::isfinite(sm_scale)))
        return fail(PKV_ERR_INVALID_ARG, "sm_scale must be finite");
    if (fp8 && (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) ||
                !std::isfinite(v_scale)))
        return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    if (num_ctas < -pkv::kMaxCluster)
        return fail(PKV_ERR_INVALID_ARG, "num_ctas must be >= %d (got %d)", -pkv::kMaxCluster,
                    num_ctas);
    if (batch == 0) return PKV_OK;
    st = check_chunks(batch, max_pages, page_size);
    if (st != PKV_OK) return st;
    if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !out || !lse ||
        (int4 && (!pools.k_params || !pools.v_params)))
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 4) ||
        !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(pools.k_params, 16) || !aligned(pools.v_params, 16))
        return fail(PKV_ERR_INVALID_ARG, "misaligned pointer (q and caches need 16 bytes)");
    // a window that covers every length the page table allows hides nothing
    if (window >= static_cast<int64_t>(max_pages) * page_size) window = sinks = 0;
    if (!workspace || !aligned(workspace, 256))
        return fail(PKV_ERR_WORKSPACE, "workspace must be non-null and 256-byte aligned");

    AttnPlan plan;
    st = plan_attention(kv, batch, num_kv_heads, group, head_dim, max_pages, page_size, window,
                        sinks, num_ctas, &plan);
    if (st != PKV_OK) return st;
    const int kv_per_item = plan.kv_per_item;
    const int grid = plan.grid;
    const int cluster = plan.cluster, nclusters = plan.nclusters;
    const pkv::WorkspaceLayout wl =
        pkv::workspace_layout(batch, group, num_kv_heads, plan.ws_kv_per_item, head_dim, grid);
    if (workspace_bytes < wl.total)
        return fail(PKV_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes,
                    wl.total);

    // rows of one TMA box: a 64-token chunk of a page (a whole page when
    // smaller); with two KV heads per item and 64-token pages (INT4: up to 64),
    // both heads' rows of the page at once (they are adjacent in the pool)
    const bool joint = kv_per_item == 2 && (page_size == pkv::kChunkTokens ||
                                            (int4 && page_size < pkv::kChunkTokens));
    const int box_rows = std::min<int>(page_size, pkv::kChunkTokens) * (joint ? 2 : 1);
    const int64_t rows = static_cast<int64_t>(num_pages) * num_kv_heads * page_size;
    CUtensorMap tk, tv;
    st = encode_pool_map(&tk, k_cache, kv, head_dim, rows, box_rows);
    if (st != PKV_OK) return st;
    st = encode_pool_map(&tv, v_cache, kv, head_dim, rows, box_rows);
    if (st != PKV_OK) return st;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    pkv::AttnArgs a{};
    a.q = q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.abort = abort;
    a.out = out;
    a.lse = lse;
    a.ws_status = reinterpret_cast<uint32_t*>(ws);
    a.ws_ml = reinterpret_cast<float*>(ws + wl.ml_off);
    a.ws_o = reinterpret_cast<float*>(ws + wl.o_off);
    a.batch = batch;
    a.max_pages = max_pages;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.kv_per_item = kv_per_item;
    a.items_per_req = num_kv_heads / kv_per_item;
    a.group = group;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.num_ctas = cluster > 0 ? cluster * nclusters : grid;
    a.box_rows = box_rows;
    a.cluster_size = cluster;
    a.num_clusters = nclusters;
    a.qk_scale = sm_scale * (fp8 ? k_scale : 1.f) * 1.4426950408889634f;
    a.v_scale = fp8 ? v_scale : 1.f;
    a.k_codes = int4 ? static_cast<const uint8_t*>(k_cache) : nullptr;
    a.v_codes = int4 ? static_cast<const uint8_t*>(v_cache) : nullptr;
    a.k_params = reinterpret_cast<const uint8_t*>(pools.k_params);
    a.v_params = reinterpret_cast<const uint8_t*>(pools.v_params);
    a.window = window;
    a.sinks = sinks;

    cudaError_t e = pkv::launch_attn_partial(
        variant_of(kv, head_dim, group, kv_per_item, window > 0), a.num_ctas, as_stream(stream),
        tk, tv, a);
    if (e != cudaSuccess) return cuda_fail(e, "attention partial launch");
    if (cluster == 0) {
        e = pkv::launch_attn_merge(head_dim, as_stream(stream), a);
        if (e != cudaSuccess) return cuda_fail(e, "attention merge launch");
    }
    return PKV_OK;
}

// Shared-prefix mode: the split-K workspace, then the prefix records and the
// plan arrays.
struct PrefixLayout {
    size_t pml_off, po_off, link_off, leader_off, refkey_off, ref_off, share_off, pshare_off,
        cbeg_off, tiles_off, ntiles_off, total;
};

bool prefix_supported(int32_t num_kv_heads, int32_t group, int32_t head_dim) {
    return head_dim == 128 && pkv::kv_heads_per_item(PKV_KV_FP8, num_kv_heads, group) == 2;
}

PrefixLayout prefix_layout(size_t base, int32_t batch, int32_t num_kv_heads, int32_t group) {
    PrefixLayout l{};
    const size_t items = static_cast<size_t>(batch) * (num_kv_heads / 2);
    const size_t heads = 2 * static_cast<size_t>(group);
    const size_t B = static_cast<size_t>(batch);
    l.pml_off = round_up(base, 256);
    l.po_off = round_up(l.pml_off + items * heads * 4 * 4, 256);
    l.link_off = round_up(l.po_off + items * heads * 128 * 4, 256);
    l.leader_off = round_up(l.link_off + B * 4, 256);
    l.refkey_off = round_up(l.leader_off + B * 4, 256);
    l.ref_off = round_up(l.refkey_off + B * 8, 256);
    l.share_off = round_up(l.ref_off + B * 4, 256);
    l.pshare_off = round_up(l.share_off + B * 4, 256);
    l.cbeg_off = round_up(l.pshare_off + B * 4, 256);
    l.tiles_off = round_up(l.cbeg_off + B * 4, 256);
    l.ntiles_off = round_up(l.tiles_off + (B / 2 + 1) * 4 * 4, 256);
    l.total = round_up(l.ntiles_off + 4, 256);
    return l;
}

pkv_status prefix_impl(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                       float k_scale, float v_scale, const int32_t* page_table, int32_t max_pages,
                       const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                       int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                       int32_t num_pages, float sm_scale, const uint8_t* abort, uint16_t* out,
                       float* lse, void* workspace, size_t workspace_bytes, int32_t num_ctas,
                       int32_t* chunk_begin_out, void* stream) {
    pkv_status st = check_common_kv(batch, num_kv_heads, head_dim, page_size, num_pages, max_pages);
    if (st != PKV_OK) return st;
    if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(PKV_ERR_INVALID_ARG, "num_q_heads (%d) must be a positive multiple of "
                    "num_kv_heads (%d)", num_q_heads, num_kv_heads);
    const int group = num_q_heads / num_kv_heads;
    if (num_ctas < 0)
        return fail(PKV_ERR_INVALID_ARG, "num_ctas must be >= 0 in shared-prefix mode (got %d)",
                    num_ctas);
    if (!prefix_supported(num_kv_heads, group, head_dim)) {
        // no shared-prefix tile for this shape: the plain call, no chunk shared
        st = attn_impl({PKV_KV_FP8, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr}, q,
                       page_table, max_pages, seq_lens, batch, num_q_heads, num_kv_heads,
                       head_dim, page_size, num_pages, sm_scale, 0, 0, abort, out, lse, workspace,
                       workspace_bytes, num_ctas, stream);
        if (st != PKV_OK || chunk_begin_out == nullptr || batch == 0) return st;
        cudaError_t e = cudaMemsetAsync(chunk_begin_out, 0, static_cast<size_t>(batch) * 4,
                                        as_stream(stream));
        return e == cudaSuccess ? PKV_OK : cuda_fail(e, "cudaMemsetAsync");
    }
    if (!(std::isfinite(sm_scale)))
        return fail(PKV_ERR_INVALID_ARG, "sm_scale must be finite");
    if (!(k_scale > 0.f) || !(v_scale > 0.f) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
        return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    if (batch == 0) return PKV_OK;
    st = check_chunks(batch, max_pages, page_size);
    if (st != PKV_OK) return st;
    if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !out || !lse)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 4) ||
        !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
        (chunk_begin_out && !aligned(chunk_begin_out, 4)))
        return fail(PKV_ERR_INVALID_ARG, "misaligned pointer (q and caches need 16 bytes)");
    if (!workspace || !aligned(workspace, 256))
        return fail(PKV_ERR_WORKSPACE, "workspace must be non-null and 256-byte aligned");

    AttnPlan plan;
    st = plan_attention(PKV_KV_FP8, batch, num_kv_heads, group, head_dim, max_pages, page_size, 0, 0,
                        num_ctas, &plan, /*allow_cluster=*/false);
    if (st != PKV_OK) return st;
    const DeviceInfo* info = nullptr;
    st = device_info(&info);
    if (st != PKV_OK) return st;
    const pkv::WorkspaceLayout wl =
        pkv::workspace_layout(batch, group, num_kv_heads, 2, head_dim, plan.grid);
    const PrefixLayout pl = prefix_layout(wl.total, batch, num_kv_heads, group);
    if (workspace_bytes < pl.total)
        return fail(PKV_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", workspace_bytes,
                    pl.total);
    int pfx_blocks = 1;   // resident shared-prefix CTAs per SM
    {
        static std::mutex m;
        static int blocks[kMaxDevices] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
        std::lock_guard<std::mutex> lock(m);
        if (blocks[dev] == 0) {
            e = pkv::prefix_set_smem_attr();
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
            int n = 0;
            e = pkv::prefix_occupancy(&n);
            if (e != cudaSuccess) return cuda_fail(e, "occupancy query");
            if (n < 1) {
                int regs = 0, local = 0, maxt = 0;
                pkv::prefix_attributes(&regs, &local, &maxt);
                return fail(PKV_ERR_UNSUPPORTED,
                            "the shared-prefix kernel does not fit on an SM of this device "
                            "(%d registers, %d local bytes per thread, at most %d threads per CTA)",
                            regs, local, maxt);
            }
            blocks[dev] = n;
        }
        pfx_blocks = blocks[dev];
    }

    const int box_rows = page_size < pkv::kChunkTokens ? page_size : pkv::kChunkTokens;
    const int64_t rows = static_cast<int64_t>(num_pages) * num_kv_heads * page_size;
    CUtensorMap tk_p, tv_p, tk, tv;
    // the prefix pass loads one head's 64 rows (or a page of them) per box
    st = encode_pool_map(&tk_p, k_cache, PKV_KV_FP8, head_dim, rows, box_rows);
    if (st != PKV_OK) return st;
    st = encode_pool_map(&tv_p, v_cache, PKV_KV_FP8, head_dim, rows, box_rows);
    if (st != PKV_OK) return st;
    // the split-K kernel's boxes (both heads of a 64-token page at once)
    const int box_rows_s = page_size == pkv::kChunkTokens ? 2 * pkv::kChunkTokens : box_rows;
    st = encode_pool_map(&tk, k_cache, PKV_KV_FP8, head_dim, rows, box_rows_s);
    if (st != PKV_OK) return st;
    st = encode_pool_map(&tv, v_cache, PKV_KV_FP8, head_dim, rows, box_rows_s);
    if (st != PKV_OK) return st;

    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const float qk_scale = sm_scale * k_scale * 1.4426950408889634f;
    pkv::PrefixArgs pa{};
    pa.q = q;
    pa.page_table = page_table;
    pa.seq_lens = seq_lens;
    pa.abort = abort;
    pa.status = reinterpret_cast<uint32_t*>(ws);
    pa.pfx_ml = reinterpret_cast<float*>(ws + pl.pml_off);
    pa.pfx_o = reinterpret_cast<float*>(ws + pl.po_off);
    pa.link = reinterpret_cast<int32_t*>(ws + pl.link_off);
    pa.leader = reinterpret_cast<int32_t*>(ws + pl.leader_off);
    pa.refkey = reinterpret_cast<unsigned long long*>(ws + pl.refkey_off);
    pa.ref = reinterpret_cast<int32_t*>(ws + pl.ref_off);
    pa.share = reinterpret_cast<int32_t*>(ws + pl.share_off);
    pa.pshare = reinterpret_cast<int32_t*>(ws + pl.pshare_off);
    pa.chunk_begin = reinterpret_cast<int32_t*>(ws + pl.cbeg_off);
    pa.tiles = reinterpret_cast<int32_t*>(ws + pl.tiles_off);
    pa.num_tiles = reinterpret_cast<int32_t*>(ws + pl.ntiles_off);
    pa.batch = batch;
    pa.max_pages = max_pages;
    pa.num_q_heads = num_q_heads;
    pa.num_kv_heads = num_kv_heads;
    pa.group = group;
    pa.page_size = page_size;
    pa.num_pages = num_pages;
    pa.box_rows = box_rows;
    pa.items_per_req = num_kv_heads / 2;
    pa.members_per_tile = 64 / group;
    pa.min_chunks = pkv::kPfxMinChunks;
    pa.tail_chunks = pkv::kPfxTailChunks;
    pa.out = out;
    pa.lse = lse;
    pa.qk_scale = qk_scale;
    pa.v_scale = v_scale;

    cudaStream_t s = as_stream(stream);
    cudaError_t e = pkv::launch_prefix_plan(s, pa);
    if (e != cudaSuccess) return cuda_fail(e, "shared-prefix plan launch");
    // one wave of tile CTAs, each looping over the tiles
    e = pkv::launch_prefix_attn(pfx_blocks * info->sms, s, tk_p, tv_p, pa);
    if (e != cudaSuccess) return cuda_fail(e, "shared-prefix attention launch");

    pkv::AttnArgs a{};
    a.q = q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.abort = abort;
    a.out = out;
    a.lse = lse;
    a.ws_status = reinterpret_cast<uint32_t*>(ws);
    a.ws_ml = reinterpret_cast<float*>(ws + wl.ml_off);
    a.ws_o = reinterpret_cast<float*>(ws + wl.o_off);
    a.batch = batch;
    a.max_pages = max_pages;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.kv_per_item = 2;
    a.items_per_req = num_kv_heads / 2;
    a.group = group;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.num_ctas = plan.grid;
    a.box_rows = box_rows_s;
    a.cluster_size = 0;
    a.num_clusters = 0;
    a.qk_scale = qk_scale;
    a.v_scale = v_scale;
    a.chunk_begin = pa.chunk_begin;
    a.pfx_ml = pa.pfx_ml;
    a.pfx_o = pa.pfx_o;
    e = pkv::launch_attn_partial(variant_of(PKV_KV_FP8, head_dim, group, 2, false), plan.grid, s, tk,
                                 tv, a);
    if (e != cudaSuccess) return cuda_fail(e, "attention partial launch");
    e = pkv::launch_attn_merge(head_dim, s, a);
    if (e != cudaSuccess) return cuda_fail(e, "attention merge launch");
    if (chunk_begin_out != nullptr) {
        e = cudaMemcpyAsync(chunk_begin_out, pa.chunk_begin, static_cast<size_t>(batch) * 4,
                            cudaMemcpyDeviceToDevice, s);
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyAsync");
    }
    return PKV_OK;
}

}  // namespace

namespace pkv {
void set_last_error(const char* message) { g_last_error = message; }

WorkspaceLayout workspace_layout(int32_t batch, int32_t group, int32_t num_kv_heads,
                                 int32_t kv_per_item, int32_t head_dim, int32_t num_ctas) {
    WorkspaceLayout l{};
    const size_t items = static_cast<size_t>(batch) * (num_kv_heads / kv_per_item);
    const size_t heads_per_slot = static_cast<size_t>(group) * kv_per_item;
    const size_t slots = static_cast<size_t>(num_ctas) + items;
    l.ml_off = 256;   // after the status word
    l.o_off = round_up(l.ml_off + slots * heads_per_slot * 4 * 4, 256);
    l.total = round_up(l.o_off + slots * heads_per_slot * head_dim * 4, 256);
    return l;
}
}  // namespace pkv

extern "C" {

const char* pkv_last_error(void) { return g_last_error.c_str(); }

int32_t pkv_version(void) { return 100; }

static pkv_status check_window(int32_t window, int32_t sinks) {
    if (window < 1) return fail(PKV_ERR_INVALID_ARG, "window must be >= 1 (got %d)", window);
    if (sinks < 0) return fail(PKV_ERR_INVALID_ARG, "sinks must be >= 0 (got %d)", sinks);
    return PKV_OK;
}

// Per-device set-up (kernel attributes) of the calls that need nothing else of it.
static pkv_status device_setup() {
    const DeviceInfo* info = nullptr;
    return device_info(&info);
}

static pkv_status tag_check_impl(const uint32_t* page_tags, int32_t num_pages,
                                 const int32_t* page_table, const uint32_t* expected_tags,
                                 int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                 int32_t page_size, int32_t window, int32_t sinks,
                                 uint8_t* abort_out, int32_t* num_aborted, void* stream) {
    if (batch < 0) return fail(PKV_ERR_INVALID_ARG, "batch must be >= 0");
    if (num_pages < 1 || max_pages < 1 || page_size < 1)
        return fail(PKV_ERR_INVALID_ARG, "num_pages, max_pages and page_size must be >= 1");
    if (batch > 0 && (!page_tags || !page_table || !expected_tags || !seq_lens || !abort_out))
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (num_aborted) {
        cudaError_t e = cudaMemsetAsync(num_aborted, 0, sizeof(int32_t), as_stream(stream));
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(num_aborted)");
    }
    if (batch == 0) return PKV_OK;
    const pkv_status ds = device_setup();
    if (ds != PKV_OK) return ds;
    cudaError_t e = pkv::launch_tag_check(page_tags, num_pages, page_table, expected_tags,
                                          max_pages, seq_lens, batch, page_size, window, sinks,
                                          abort_out, num_aborted, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tag check launch");
    return PKV_OK;
}

pkv_status kv_tag_check(const uint32_t* page_tags, int32_t num_pages, const int32_t* page_table,
                        const uint32_t* expected_tags, int32_t max_pages, const int32_t* seq_lens,
                        int32_t batch, int32_t page_size, uint8_t* abort_out,
                        int32_t* num_aborted, void* stream) {
    return tag_check_impl(page_tags, num_pages, page_table, expected_tags, max_pages, seq_lens,
                          batch, page_size, 0, 0, abort_out, num_aborted, stream);
}

pkv_status kv_tag_check_window(const uint32_t* page_tags, int32_t num_pages,
                               const int32_t* page_table, const uint32_t* expected_tags,
                               int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                               int32_t page_size, int32_t window, int32_t sinks,
                               uint8_t* abort_out, int32_t* num_aborted, void* stream) {
    const pkv_status st = check_window(window, sinks);
    if (st != PKV_OK) return st;
    return tag_check_impl(page_tags, num_pages, page_table, expected_tags, max_pages, seq_lens,
                          batch, page_size, window, sinks, abort_out, num_aborted, stream);
}

// The scales of an FP8 cache, and the pools of any cache (non-null, aligned).
static pkv_status check_scales(const pkv::KvDst& c) {
    if (c.kv == PKV_KV_FP8 && (!(c.k_scale > 0.f) || !(c.v_scale > 0.f) ||
                               !std::isfinite(c.k_scale) || !std::isfinite(c.v_scale)))
        return fail(PKV_ERR_INVALID_ARG, "k_scale and v_scale must be finite and > 0");
    return PKV_OK;
}
static pkv_status check_pools(const pkv::KvDst& c) {
    if (!c.k || !c.v || (c.kv == PKV_KV_INT4 && (!c.k_params || !c.v_params)))
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_params, 16) ||
        !aligned(c.v_params, 16))
        return fail(PKV_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
    return PKV_OK;
}

static pkv::KvDst fp8_pools(const uint8_t* k, const uint8_t* v, float k_scale, float v_scale) {
    return {PKV_KV_FP8, const_cast<uint8_t*>(k), const_cast<uint8_t*>(v), k_scale, v_scale,
            nullptr, nullptr};
}
static pkv::KvDst bf16_pools(const uint16_t* k, const uint16_t* v) {
    return {PKV_KV_BF16, const_cast<uint16_t*>(k), const_cast<uint16_t*>(v), 1.f, 1.f,
            nullptr, nullptr};
}
static pkv::KvDst int4_pools(const uint8_t* k, const uint16_t* kp, const uint8_t* v,
                             const uint16_t* vp) {
    return {PKV_KV_INT4, const_cast<uint8_t*>(k), const_cast<uint8_t*>(v), 1.f, 1.f,
            reinterpret_cast<uint32_t*>(const_cast<uint16_t*>(kp)),
            reinterpret_cast<uint32_t*>(const_cast<uint16_t*>(vp))};
}

static pkv_status append_impl(const pkv::KvDst& dst, const uint16_t* k_new, const uint16_t* v_new,
                              const int32_t* page_table, int32_t max_pages,
                              const int32_t* seq_lens, int32_t batch, int32_t num_kv_heads,
                              int32_t head_dim, int32_t page_size, int32_t num_pages,
                              const uint8_t* abort, void* stream) {
    pkv_status st = check_common_kv(batch, num_kv_heads, head_dim, page_size, num_pages, max_pages);
    if (st == PKV_OK) st = check_scales(dst);
    if (st != PKV_OK) return st;
    if (batch == 0) return PKV_OK;
    if (!k_new || !v_new || !page_table || !seq_lens)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    st = check_pools(dst);
    if (st != PKV_OK) return st;
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    st = device_setup();
    if (st != PKV_OK) return st;
    cudaError_t e = pkv::launch_append(dst, k_new, v_new, page_table, max_pages, seq_lens, batch,
                                       num_kv_heads, head_dim, page_size, num_pages, abort,
                                       as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "append launch");
    return PKV_OK;
}

pkv_status kv_append_fp8(const uint16_t* k_new, const uint16_t* v_new, const int32_t* page_table,
                         int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                         int32_t num_kv_heads, int32_t head_dim, int32_t page_size, float k_scale,
                         float v_scale, uint8_t* k_cache, uint8_t* v_cache, int32_t num_pages,
                         const uint8_t* abort, void* stream) {
    return append_impl(fp8_pools(k_cache, v_cache, k_scale, v_scale), k_new, v_new, page_table,
                       max_pages, seq_lens, batch, num_kv_heads, head_dim, page_size, num_pages,
                       abort, stream);
}

pkv_status kv_append_bf16(const uint16_t* k_new, const uint16_t* v_new,
                          const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                          int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                          int32_t page_size, uint16_t* k_cache, uint16_t* v_cache,
                          int32_t num_pages, const uint8_t* abort, void* stream) {
    return append_impl(bf16_pools(k_cache, v_cache), k_new, v_new, page_table, max_pages,
                       seq_lens, batch, num_kv_heads, head_dim, page_size, num_pages, abort,
                       stream);
}

pkv_status kv_append_int4(const uint16_t* k_new, const uint16_t* v_new,
                          const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                          int32_t batch, int32_t num_kv_heads, int32_t head_dim,
                          int32_t page_size, uint8_t* k_codes, uint16_t* k_params,
                          uint8_t* v_codes, uint16_t* v_params, int32_t num_pages,
                          const uint8_t* abort, void* stream) {
    return append_impl(int4_pools(k_codes, k_params, v_codes, v_params), k_new, v_new, page_table,
                       max_pages, seq_lens, batch, num_kv_heads, head_dim, page_size, num_pages,
                       abort, stream);
}

static pkv_status check_append_impl(const pkv::KvDst& dst, const uint32_t* page_tags,
                                    int32_t num_pages, const int32_t* page_table,
                                    const uint32_t* expected_tags, int32_t max_pages,
                                    const int32_t* seq_lens, int32_t batch, int32_t page_size,
                                    const uint16_t* k_new, const uint16_t* v_new,
                                    int32_t num_kv_heads, int32_t head_dim, uint8_t* abort_out,
                                    int32_t* num_aborted, void* stream) {
    pkv_status st = check_common_kv(batch, num_kv_heads, head_dim, page_size, num_pages, max_pages);
    if (st == PKV_OK) st = check_scales(dst);
    if (st != PKV_OK) return st;
    if (num_aborted) {
        cudaError_t e = cudaMemsetAsync(num_aborted, 0, sizeof(int32_t), as_stream(stream));
        if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(num_aborted)");
    }
    if (batch == 0) return PKV_OK;
    if (!page_tags || !page_table || !expected_tags || !seq_lens || !k_new || !v_new || !abort_out)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    st = check_pools(dst);
    if (st != PKV_OK) return st;
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
        return fail(PKV_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    st = device_setup();
    if (st != PKV_OK) return st;
    cudaError_t e = pkv::launch_check_append(dst, page_tags, num_pages, page_table, expected_tags,
                                             max_pages, seq_lens, batch, page_size, k_new, v_new,
                                             num_kv_heads, head_dim, abort_out, num_aborted,
                                             as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "check+append launch");
    return PKV_OK;
}

pkv_status kv_check_append_fp8(const uint32_t* page_tags, int32_t num_pages,
                               const int32_t* page_table, const uint32_t* expected_tags,
                               int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                               int32_t page_size, const uint16_t* k_new, const uint16_t* v_new,
                               int32_t num_kv_heads, int32_t head_dim, float k_scale,
                               float v_scale, uint8_t* k_cache, uint8_t* v_cache,
                               uint8_t* abort_out, int32_t* num_aborted, void* stream) {
    return check_append_impl(fp8_pools(k_cache, v_cache, k_scale, v_scale), page_tags, num_pages,
                             page_table, expected_tags, max_pages, seq_lens, batch, page_size,
                             k_new, v_new, num_kv_heads, head_dim, abort_out, num_aborted, stream);
}

pkv_status kv_check_append_bf16(const uint32_t* page_tags, int32_t num_pages,
                                const int32_t* page_table, const uint32_t* expected_tags,
                                int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                int32_t page_size, const uint16_t* k_new, const uint16_t* v_new,
                                int32_t num_kv_heads, int32_t head_dim, uint16_t* k_cache,
                                uint16_t* v_cache, uint8_t* abort_out, int32_t* num_aborted,
                                void* stream) {
    return check_append_impl(bf16_pools(k_cache, v_cache), page_tags, num_pages, page_table,
                             expected_tags, max_pages, seq_lens, batch, page_size, k_new, v_new,
                             num_kv_heads, head_dim, abort_out, num_aborted, stream);
}

pkv_status kv_check_append_int4(const uint32_t* page_tags, int32_t num_pages,
                                const int32_t* page_table, const uint32_t* expected_tags,
                                int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                int32_t page_size, const uint16_t* k_new, const uint16_t* v_new,
                                int32_t num_kv_heads, int32_t head_dim, uint8_t* k_codes,
                                uint16_t* k_params, uint8_t* v_codes, uint16_t* v_params,
                                uint8_t* abort_out, int32_t* num_aborted, void* stream) {
    return check_append_impl(int4_pools(k_codes, k_params, v_codes, v_params), page_tags,
                             num_pages, page_table, expected_tags, max_pages, seq_lens, batch,
                             page_size, k_new, v_new, num_kv_heads, head_dim, abort_out,
                             num_aborted, stream);
}

// One token write (out == false) or read (out == true) by slot map.
static pkv_status slots_impl(const pkv::KvDst& pools, bool out, const uint16_t* k,
                             const uint16_t* v, int64_t k_stride, int64_t v_stride,
                             const int32_t* slot_map, int32_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size, int32_t num_pages,
                             void* stream) {
    pkv_status st = check_common_kv(num_tokens, num_kv_heads, head_dim, page_size, num_pages, 1);
    if (st == PKV_OK) st = check_scales(pools);
    if (st != PKV_OK) return st;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return fail(PKV_ERR_INVALID_ARG,
                    "token strides must be multiples of 8 and at least num_kv_heads * head_dim");
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_map) return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    st = check_pools(pools);
    if (st != PKV_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4))
        return fail(PKV_ERR_INVALID_ARG, "the token rows must be 16-byte aligned");
    const pkv::SlotArgs a{slot_map, num_tokens, num_kv_heads, head_dim, page_size, num_pages,
                          k_stride, v_stride};
    cudaError_t e = out ? pkv::launch_read_slots(pools, const_cast<uint16_t*>(k),
                                                 const_cast<uint16_t*>(v), a, as_stream(stream))
                        : pkv::launch_write_slots(pools, k, v, a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, out ? "slot read launch" : "slot write launch");
    return PKV_OK;
}

pkv_status kv_write_slots_fp8(const uint16_t* k_new, const uint16_t* v_new, int64_t k_stride,
                              int64_t v_stride, const int32_t* slot_map, int32_t num_tokens,
                              int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                              float k_scale, float v_scale, uint8_t* k_cache, uint8_t* v_cache,
                              int32_t num_pages, void* stream) {
    return slots_impl(fp8_pools(k_cache, v_cache, k_scale, v_scale), false, k_new, v_new, k_stride,
                      v_stride, slot_map, num_tokens, num_kv_heads, head_dim, page_size, num_pages,
                      stream);
}

pkv_status kv_write_slots_bf16(const uint16_t* k_new, const uint16_t* v_new, int64_t k_stride,
                               int64_t v_stride, const int32_t* slot_map, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               uint16_t* k_cache, uint16_t* v_cache, int32_t num_pages,
                               void* stream) {
    return slots_impl(bf16_pools(k_cache, v_cache), false, k_new, v_new, k_stride, v_stride,
                      slot_map, num_tokens, num_kv_heads, head_dim, page_size, num_pages, stream);
}

pkv_status kv_write_slots_int4(const uint16_t* k_new, const uint16_t* v_new, int64_t k_stride,
                               int64_t v_stride, const int32_t* slot_map, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                               uint8_t* k_codes, uint16_t* k_params, uint8_t* v_codes,
                               uint16_t* v_params, int32_t num_pages, void* stream) {
    return slots_impl(int4_pools(k_codes, k_params, v_codes, v_params), false, k_new, v_new,
                      k_stride, v_stride, slot_map, num_tokens, num_kv_heads, head_dim, page_size,
                      num_pages, stream);
}

pkv_status kv_read_slots_fp8(const int32_t* slot_map, int32_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int32_t page_size, float k_scale, float v_scale,
                             const uint8_t* k_cache, const uint8_t* v_cache, int32_t num_pages,
                             uint16_t* k_out, uint16_t* v_out, int64_t k_stride, int64_t v_stride,
                             void* stream) {
    return slots_impl(fp8_pools(k_cache, v_cache, k_scale, v_scale), true, k_out, v_out, k_stride,
                      v_stride, slot_map, num_tokens, num_kv_heads, head_dim, page_size, num_pages,
                      stream);
}

pkv_status kv_read_slots_bf16(const int32_t* slot_map, int32_t num_tokens, int32_t num_kv_heads,
                              int32_t head_dim, int32_t page_size, const uint16_t* k_cache,
                              const uint16_t* v_cache, int32_t num_pages, uint16_t* k_out,
                              uint16_t* v_out, int64_t k_stride, int64_t v_stride, void* stream) {
    return slots_impl(bf16_pools(k_cache, v_cache), true, k_out, v_out, k_stride, v_stride,
                      slot_map, num_tokens, num_kv_heads, head_dim, page_size, num_pages, stream);
}

pkv_status kv_read_slots_int4(const int32_t* slot_map, int32_t num_tokens, int32_t num_kv_heads,
                              int32_t head_dim, int32_t page_size, const uint8_t* k_codes,
                              const uint16_t* k_params, const uint8_t* v_codes,
                              const uint16_t* v_params, int32_t num_pages, uint16_t* k_out,
                              uint16_t* v_out, int64_t k_stride, int64_t v_stride, void* stream) {
    return slots_impl(int4_pools(k_codes, k_params, v_codes, v_params), true, k_out, v_out,
                      k_stride, v_stride, slot_map, num_tokens, num_kv_heads, head_dim, page_size,
                      num_pages, stream);
}

pkv_status kv_extend_tables(const int32_t* old_lens, const int32_t* new_lens, int32_t batch,
                            int32_t page_size, const int32_t* free_pages, int32_t free_capacity,
                            const int32_t* num_free, int32_t* num_free_out, int32_t num_pages,
                            int32_t* page_table, int32_t max_pages, const uint32_t* page_tags,
                            uint32_t* expected_tags, int32_t* slot_map, int32_t max_tokens,
                            int32_t* cu_tokens, uint8_t* failed, void* stream) {
    if (batch < 0 || max_tokens < 0 || free_capacity < 0)
        return fail(PKV_ERR_INVALID_ARG, "batch, max_tokens and free_capacity must be >= 0");
    if (num_pages < 1 || max_pages < 1)
        return fail(PKV_ERR_INVALID_ARG, "num_pages and max_pages must be >= 1");
    if (!supported_page_size(page_size))
        return fail(PKV_ERR_UNSUPPORTED, "page_size %d not supported (16, 32, 64 or 128)", page_size);
    if (static_cast<int64_t>(num_pages) * page_size > INT32_MAX)
        return fail(PKV_ERR_UNSUPPORTED, "num_pages * page_size must be < 2^31");
    if (free_capacity > num_pages)
        return fail(PKV_ERR_INVALID_ARG, "free_capacity must be at most num_pages");
    if ((page_tags == nullptr) != (expected_tags == nullptr))
        return fail(PKV_ERR_INVALID_ARG, "page_tags and expected_tags are given together or neither is");
    if (!num_free || !num_free_out || !cu_tokens || (free_capacity > 0 && !free_pages) ||
        (max_tokens > 0 && !slot_map) ||
        (batch > 0 && (!old_lens || !new_lens || !page_table || !failed)))
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    const void* words[] = {old_lens, new_lens,      free_pages, num_free, num_free_out, page_table,
                           page_tags, expected_tags, slot_map,   cu_tokens};
    for (const void* p : words)
        if (!aligned(p, 4)) return fail(PKV_ERR_INVALID_ARG, "misaligned pointer");
    const pkv::TableArgs a{old_lens,  new_lens,  free_pages,    num_free,  num_free_out, page_table,
                           page_tags, expected_tags, cu_tokens, slot_map,  failed,       batch,
                           page_size, free_capacity, num_pages, max_pages, max_tokens};
    cudaError_t e = pkv::launch_extend_tables(a, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "extend tables launch");
    return PKV_OK;
}

pkv_status kv_retag_pages(uint32_t* page_tags, int32_t num_pages, const int32_t* pages,
                          int32_t num_ids, void* stream) {
    if (num_pages < 1 || num_ids < 0)
        return fail(PKV_ERR_INVALID_ARG, "num_pages must be >= 1 and num_ids >= 0");
    if (num_ids == 0) return PKV_OK;
    if (!page_tags || !pages) return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(page_tags, 4) || !aligned(pages, 4))
        return fail(PKV_ERR_INVALID_ARG, "misaligned pointer");
    cudaError_t e = pkv::launch_retag(page_tags, num_pages, pages, num_ids, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "retag launch");
    return PKV_OK;
}

pkv_status kv_expected_tags(const uint32_t* page_tags, int32_t num_pages,
                            const int32_t* page_table, int32_t max_pages,
                            const int32_t* seq_lens, int32_t batch, int32_t page_size,
                            uint32_t* expected_tags, void* stream) {
    if (batch < 0 || num_pages < 1 || max_pages < 1 || page_size < 1)
        return fail(PKV_ERR_INVALID_ARG, "invalid sizes");
    if (batch == 0) return PKV_OK;
    if (!page_tags || !page_table || !seq_lens || !expected_tags)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    cudaError_t e = pkv::launch_expected_tags(page_tags, num_pages, page_table, max_pages,
                                              seq_lens, batch, page_size, expected_tags,
                                              as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "expected-tags launch");
    return PKV_OK;
}

// The sizes of a page handoff.
static pkv_status check_requant(int32_t src_num_pages, int32_t dst_num_pages, int32_t num_pairs,
                                int32_t num_kv_heads, int32_t page_size, int32_t head_dim) {
    if (num_pairs < 0) return fail(PKV_ERR_INVALID_ARG, "num_pairs must be >= 0");
    if (src_num_pages < 1 || dst_num_pages < 1 || num_kv_heads < 1)
        return fail(PKV_ERR_INVALID_ARG, "pool sizes and num_kv_heads must be >= 1");
    if (!supported_head_dim(head_dim))
        return fail(PKV_ERR_UNSUPPORTED, "head_dim %d not supported (64 or 128)", head_dim);
    if (!supported_page_size(page_size))
        return fail(PKV_ERR_UNSUPPORTED, "page_size %d not supported", page_size);
    return PKV_OK;
}

pkv_status kv_requant_pages_fp8(const uint16_t* src_pool, int32_t src_num_pages,
                                const int32_t* src_pages, uint8_t* dst_pool,
                                int32_t dst_num_pages, const int32_t* dst_pages,
                                int32_t num_pairs, int32_t num_kv_heads, int32_t page_size,
                                int32_t head_dim, float scale, void* stream) {
    const pkv_status st = check_requant(src_num_pages, dst_num_pages, num_pairs, num_kv_heads,
                                        page_size, head_dim);
    if (st != PKV_OK) return st;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return fail(PKV_ERR_INVALID_ARG, "scale must be finite and > 0");
    if (num_pairs == 0) return PKV_OK;
    if (!src_pool || !src_pages || !dst_pool || !dst_pages)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(src_pool, 16) || !aligned(dst_pool, 16))
        return fail(PKV_ERR_INVALID_ARG, "pools must be 16-byte aligned");
    const int64_t page_elems = static_cast<int64_t>(num_kv_heads) * page_size * head_dim;
    cudaError_t e = pkv::launch_requant(src_pool, src_num_pages, src_pages, dst_pool,
                                        dst_num_pages, dst_pages, num_pairs, page_elems, scale,
                                        as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "requant launch");
    return PKV_OK;
}

pkv_status kv_requant_pages_int4(const uint16_t* src_pool, int32_t src_num_pages,
                                 const int32_t* src_pages, uint8_t* dst_codes,
                                 uint16_t* dst_params, int32_t dst_num_pages,
                                 const int32_t* dst_pages, int32_t num_pairs,
                                 int32_t num_kv_heads, int32_t page_size, int32_t head_dim,
                                 void* stream) {
    const pkv_status st = check_requant(src_num_pages, dst_num_pages, num_pairs, num_kv_heads,
                                        page_size, head_dim);
    if (st != PKV_OK) return st;
    if (num_pairs == 0) return PKV_OK;
    if (!src_pool || !src_pages || !dst_codes || !dst_params || !dst_pages)
        return fail(PKV_ERR_INVALID_ARG, "null pointer argument");
    if (!aligned(src_pool, 16) || !aligned(dst_codes, 16) || !aligned(dst_params, 16))
        return fail(PKV_ERR_INVALID_ARG, "pools must be 16-byte aligned");
    const int64_t page_elems = static_cast<int64_t>(num_kv_heads) * page_size * head_dim;
    cudaError_t e = pkv::launch_requant_int4(src_pool, src_num_pages, src_pages, dst_codes,
                                             reinterpret_cast<uint32_t*>(dst_params),
                                             dst_num_pages, dst_pages, num_pairs, page_elems,
                                             head_dim, as_stream(stream));
    if (e != cudaSuccess) return cuda_fail(e, "requant launch");
    return PKV_OK;
}

pkv_status paged_decode_attn_plan(int32_t kv_dtype, int32_t batch, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, int32_t max_pages,
                                  int32_t page_size, int32_t num_ctas, int32_t* cluster_size,
                                  int32_t* ctas, int32_t* launches) {
    if (!known_kv(kv_dtype))
        return fail(PKV_ERR_INVALID_ARG, "kv_dtype must be PKV_KV_FP8, PKV_KV_BF16 or PKV_KV_INT4");
    if (!cluster_size || !ctas || !launches)
        return fail(PKV_ERR_INVALID_ARG, "null output pointer");
    if (batch < 1) return fail(PKV_ERR_INVALID_ARG, "batch must be >= 1");
    pkv_status st = check_common_kv(batch, num_kv_heads, head_dim, page_size, 1, max_pages);
    if (st != PKV_OK) return st;
    if (num_q_heads < 1 || num_q_heads % num_kv_heads != 0)
        return fail(PKV_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
    const int group = num_q_heads / num_kv_heads;
    if (group > 16) return fail(PKV_ERR_UNSUPPORTED, "GQA group %d > 16 not supported", group);
    if (num_ctas < -pkv::kMaxCluster)
        return fail(PKV_ERR_INVALID_ARG, "num_ctas must be >= %d", -pkv::kMaxCluster);
    st = check_chunks(batch, max_pages, page_size);
    if (st != PKV_OK) return st;
    AttnPlan plan;
    st = plan_attention(kv_dtype, batch, num_kv_heads, group, head_dim, max_pages, page_size, 0, 0,
                        num_ctas, &plan);
    if (st != PKV_OK) return st;
    *cluster_size = plan.cluster;
    *ctas = plan.cluster > 0 ? plan.cluster * plan.nclusters : plan.grid;
    *launches = plan.cluster > 0 ? 1 : 2;
    return PKV_OK;
}

size_t paged_decode_attn_workspace_size(int32_t kv_dtype, int32_t batch, int32_t num_q_heads,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t num_ctas) {
    if (!known_kv(kv_dtype)) {
        fail(PKV_ERR_INVALID_ARG, "kv_dtype must be PKV_KV_FP8, PKV_KV_BF16 or PKV_KV_INT4");
        return 0;
    }
    if (batch < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        !supported_head_dim(head_dim) || num_ctas < -pkv::kMaxCluster) {
        fail(PKV_ERR_INVALID_ARG, "invalid sizes for the workspace query");
        return 0;
    }
    const int group = num_q_heads / num_kv_heads;
    if (group > 16) {
        fail(PKV_ERR_UNSUPPORTED, "GQA group %d > 16 not supported", group);
        return 0;
    }
    int grid = num_ctas > 0 ? num_ctas : 0;   // cluster mode (< 0) needs no more than the default
    const int kv_per_item = pkv::kv_heads_per_item(kv_dtype, num_kv_heads, group);
    if (grid == 0) {
        // the larger of the grids without and with a window: one workspace serves both calls
        for (const bool window : {false, true}) {
            const auto v = variant_of(kv_dtype, head_dim, group, kv_per_item, window);
            int ctas = 0;
            if (default_ctas(v, &ctas) != PKV_OK) return 0;
            grid = std::max(grid, ctas);
        }
    }
    return pkv::workspace_layout(batch, group, num_kv_heads, kv_per_item, head_dim, grid).total;
}

pkv_status paged_decode_attn_fp8(const uint16_t* q, const uint8_t* k_cache,
                                 const uint8_t* v_cache, float k_scale, float v_scale,
                                 const int32_t* page_table, int32_t max_pages,
                                 const int32_t* seq_lens, int32_t batch, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t page_size,
                                 int32_t num_pages, float sm_scale, const uint8_t* abort,
                                 uint16_t* out, float* lse, void* workspace,
                                 size_t workspace_bytes, int32_t num_ctas, void* stream) {
    return attn_impl({PKV_KV_FP8, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr}, q,
                     page_table, max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim,
                     page_size, num_pages, sm_scale, 0, 0, abort, out, lse, workspace,
                     workspace_bytes, num_ctas, stream);
}

size_t paged_decode_attn_fp8_prefix_workspace_size(int32_t batch, int32_t num_q_heads,
                                                   int32_t num_kv_heads, int32_t head_dim,
                                                   int32_t num_ctas) {
    if (batch < 0 || num_kv_heads < 1 || num_q_heads < 1 || num_q_heads % num_kv_heads != 0 ||
        !supported_head_dim(head_dim) || num_ctas < 0) {
        fail(PKV_ERR_INVALID_ARG, "invalid sizes for the shared-prefix workspace query");
        return 0;
    }
    const int group = num_q_heads / num_kv_heads;
    if (!prefix_supported(num_kv_heads, group, head_dim))
        return paged_decode_attn_workspace_size(PKV_KV_FP8, batch, num_q_heads, num_kv_heads,
                                                head_dim, num_ctas);
    int grid = num_ctas;
    if (grid == 0 &&
        default_ctas(variant_of(PKV_KV_FP8, head_dim, group, 2, false), &grid) != PKV_OK)
        return 0;
    const size_t base = pkv::workspace_layout(batch, group, num_kv_heads, 2, head_dim, grid).total;
    return prefix_layout(base, batch, num_kv_heads, group).total;
}

pkv_status paged_decode_attn_fp8_prefix(const uint16_t* q, const uint8_t* k_cache,
                                        const uint8_t* v_cache, float k_scale, float v_scale,
                                        const int32_t* page_table, int32_t max_pages,
                                        const int32_t* seq_lens, int32_t batch,
                                        int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t page_size, int32_t num_pages,
                                        float sm_scale, const uint8_t* abort, uint16_t* out,
                                        float* lse, void* workspace, size_t workspace_bytes,
                                        int32_t num_ctas, int32_t* chunk_begin_out,
                                        void* stream) {
    return prefix_impl(q, k_cache, v_cache, k_scale, v_scale, page_table, max_pages, seq_lens,
                       batch, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale,
                       abort, out, lse, workspace, workspace_bytes, num_ctas, chunk_begin_out,
                       stream);
}

pkv_status paged_decode_attn_bf16(const uint16_t* q, const uint16_t* k_cache,
                                  const uint16_t* v_cache, const int32_t* page_table,
                                  int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t page_size, int32_t num_pages, float sm_scale,
                                  const uint8_t* abort, uint16_t* out, float* lse,
                                  void* workspace, size_t workspace_bytes, int32_t num_ctas,
                                  void* stream) {
    return attn_impl({PKV_KV_BF16, k_cache, v_cache, 1.f, 1.f, nullptr, nullptr}, q, page_table,
                     max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size,
                     num_pages, sm_scale, 0, 0, abort, out, lse, workspace, workspace_bytes,
                     num_ctas, stream);
}

pkv_status paged_decode_attn_int4(const uint16_t* q, const uint8_t* k_codes,
                                  const uint16_t* k_params, const uint8_t* v_codes,
                                  const uint16_t* v_params, const int32_t* page_table,
                                  int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t page_size, int32_t num_pages, float sm_scale,
                                  const uint8_t* abort, uint16_t* out, float* lse, void* workspace,
                                  size_t workspace_bytes, int32_t num_ctas, void* stream) {
    return attn_impl({PKV_KV_INT4, k_codes, v_codes, 1.f, 1.f, k_params, v_params}, q, page_table,
                     max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size,
                     num_pages, sm_scale, 0, 0, abort, out, lse, workspace, workspace_bytes,
                     num_ctas, stream);
}

pkv_status paged_decode_attn_fp8_window(const uint16_t* q, const uint8_t* k_cache,
                                        const uint8_t* v_cache, float k_scale, float v_scale,
                                        const int32_t* page_table, int32_t max_pages,
                                        const int32_t* seq_lens, int32_t batch,
                                        int32_t num_q_heads, int32_t num_kv_heads,
                                        int32_t head_dim, int32_t page_size, int32_t num_pages,
                                        float sm_scale, int32_t window, int32_t sinks,
                                        const uint8_t* abort, uint16_t* out, float* lse,
                                        void* workspace, size_t workspace_bytes, int32_t num_ctas,
                                        void* stream) {
    const pkv_status st = check_window(window, sinks);
    if (st != PKV_OK) return st;
    return attn_impl({PKV_KV_FP8, k_cache, v_cache, k_scale, v_scale, nullptr, nullptr}, q,
                     page_table, max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim,
                     page_size, num_pages, sm_scale, window, sinks, abort, out, lse, workspace,
                     workspace_bytes, num_ctas, stream);
}

pkv_status paged_decode_attn_bf16_window(const uint16_t* q, const uint16_t* k_cache,
                                         const uint16_t* v_cache, const int32_t* page_table,
                                         int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                         int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t page_size, int32_t num_pages,
                                         float sm_scale, int32_t window, int32_t sinks,
                                         const uint8_t* abort, uint16_t* out, float* lse,
                                         void* workspace, size_t workspace_bytes, int32_t num_ctas,
                                         void* stream) {
    const pkv_status st = check_window(window, sinks);
    if (st != PKV_OK) return st;
    return attn_impl({PKV_KV_BF16, k_cache, v_cache, 1.f, 1.f, nullptr, nullptr}, q, page_table,
                     max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size,
                     num_pages, sm_scale, window, sinks, abort, out, lse, workspace,
                     workspace_bytes, num_ctas, stream);
}

pkv_status paged_decode_attn_int4_window(const uint16_t* q, const uint8_t* k_codes,
                                         const uint16_t* k_params, const uint8_t* v_codes,
                                         const uint16_t* v_params, const int32_t* page_table,
                                         int32_t max_pages, const int32_t* seq_lens, int32_t batch,
                                         int32_t num_q_heads, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t page_size, int32_t num_pages,
                                         float sm_scale, int32_t window, int32_t sinks,
                                         const uint8_t* abort, uint16_t* out, float* lse,
                                         void* workspace, size_t workspace_bytes, int32_t num_ctas,
                                         void* stream) {
    const pkv_status st = check_window(window, sinks);
    if (st != PKV_OK) return st;
    return attn_impl({PKV_KV_INT4, k_codes, v_codes, 1.f, 1.f, k_params, v_params}, q, page_table,
                     max_pages, seq_lens, batch, num_q_heads, num_kv_heads, head_dim, page_size,
                     num_pages, sm_scale, window, sinks, abort, out, lse, workspace,
                     workspace_bytes, num_ctas, stream);
}

pkv_status int4_dequant_gemv(const uint16_t* x, const uint8_t* w_tiles, const uint16_t* scales,
                             int32_t batch, int32_t n, int32_t k, int32_t group_size, uint16_t* y,
                             uint32_t* status, void* stream) {
    if (!x || !w_tiles || !scales || !y)
        return fail(PKV_ERR_INVALID_ARG, "x, w_tiles, scales and y must be non-null");
    if (!aligned(x, 16) || !aligned(w_tiles, 16) || !aligned(scales, 16) || !aligned(y, 2) ||
        (status && !aligned(status, 4)))
        return fail(PKV_ERR_INVALID_ARG,
                    "misaligned pointer (x, w_tiles and scales need 16 bytes, y 2, status 4)");
    if (batch < 1 || batch > pkv::kGemvMaxBatch)
        return fail(PKV_ERR_INVALID_ARG, "batch must be in [1, %d] (got %d)", pkv::kGemvMaxBatch,
                    batch);
    if (n < pkv::kGemvRows || n % pkv::kGemvRows != 0)
        return fail(PKV_ERR_INVALID_ARG, "n must be a positive multiple of %d (got %d)",
                    pkv::kGemvRows, n);
    if (k < pkv::kGemvKTile || k % pkv::kGemvKTile != 0)
        return fail(PKV_ERR_INVALID_ARG, "k must be a positive multiple of %d (got %d)",
                    pkv::kGemvKTile, k);
    if (group_size != pkv::kGemvGroup)
        return fail(PKV_ERR_UNSUPPORTED, "group_size %d not supported (%d)", group_size,
                    pkv::kGemvGroup);

    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    // batches up to 16 on the warp-level MMA kernel, larger ones on tcgen05
    const bool small = batch <= pkv::kGemvMmaMaxBatch;
    const int xrows = small ? 8 * pkv::gemv_mma_batch_blocks(batch) : pkv::gemv_batch_cols(batch);
    {
        static std::mutex m;
        static bool ready[kMaxDevices][5] = {};
        const int slot = small ? (xrows == 8 ? 0 : 1) : (xrows == 16 ? 2 : (xrows == 32 ? 3 : 4));
        if (dev < 0 || dev >= kMaxDevices) return fail(PKV_ERR_UNSUPPORTED, "device %d", dev);
        std::lock_guard<std::mutex> lock(m);
        if (!ready[dev][slot]) {
            e = small ? pkv::gemv_mma_set_smem_attr(xrows / 8) : pkv::gemv_set_smem_attr(xrows);
            if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
            ready[dev][slot] = true;
        }
    }

    // codes: the tiles as rows of 128 bytes (one box = one 128 x 256 tile);
    // x: [batch][k] bf16, 64-column x xrows-row boxes (rows past batch read
    // as zero); scales: rows of 128 (one row block, one group), 2-row boxes
    CUtensorMap tw, tx, ts;
    pkv_status st = encode_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w_tiles, pkv::kGemvKTile / 2,
                              static_cast<uint64_t>(n) * (k / pkv::kGemvKTile),
                              pkv::kGemvKTile / 2, pkv::kGemvKTile / 2, pkv::kGemvRows,
                              CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != PKV_OK) return st;
    st = encode_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, static_cast<uint64_t>(k),
                   static_cast<uint64_t>(batch), static_cast<uint64_t>(k) * 2, 64, xrows,
                   CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != PKV_OK) return st;
    st = encode_2d(&ts, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, scales, pkv::kGemvRows,
                   static_cast<uint64_t>(n / pkv::kGemvRows) * (k / group_size),
                   pkv::kGemvRows * 2, pkv::kGemvRows, pkv::kGemvKTile / pkv::kGemvGroup,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != PKV_OK) return st;

    pkv::GemvArgs a{};
    a.y = y;
    a.status = status;
    a.batch = batch;
    a.n = n;
    a.k = k;
    e = small ? pkv::launch_int4_gemv_mma(xrows / 8, as_stream(stream), tw, tx, ts, a)
              : pkv::launch_int4_gemv(xrows, as_stream(stream), tw, tx, ts, a);
    if (e != cudaSuccess) return cuda_fail(e, "int4_dequant_gemv launch");
    return PKV_OK;
}

}  // extern "C"
