// kv_slots.cu -- token writes into cache slots named by a slot map, and reads
// of such slots back as bf16, for FP8, BF16 and INT4 caches.
//
// A warp moves the K row or the V row of a token, 32 consecutive 8-value blocks
// (16 bytes of bf16) at a time, or of as many consecutive tokens as fill its
// lanes; an INT4 group of 64 dims is 8 consecutive lanes, whose minimum and maximum
// meet in three shuffles.  Nothing is read twice, so memory bounds large calls,
// and the chain of two dependent loads, slot then row, small ones: up to four
// blocks of a long row are in a lane's flight together, and K and V are different
// warps.  (More rows a warp for more blocks in flight made short rows slower:
// 20,000 tokens of 1 x 64, INT4 6.0 us with four, 4.4 with one.)
#include "kv_codec.cuh"

namespace pkv {

constexpr int kSlotThreads = 256;
constexpr int kSlotWarps = kSlotThreads / 32;
// blocks of a lane in flight
template <bool kOne>
constexpr int kFlight = kOne ? 4 : 1;

// The calling warp's part of a call: blocks [0, total) of its tokens' rows.
// kOne: a single token, whose slot is loaded and resolved once (8,192 tokens of
// 8 x 128, INT4: write 16.6 us, read 9.6; block by block 18.8 and 11.7).
template <int kD, bool kOne>
struct SlotWork {
    const SlotArgs& a;
    int blocks;       // per row, a multiple of 8
    uint32_t inv;     // ceil(2^16 / blocks)
    int64_t token0;
    int total;
    bool is_v;
    int shift;        // log2(page size)
    int32_t row0;     // kOne: the token's pool row of head 0, negative without a slot

    __device__ __forceinline__ SlotWork(const SlotArgs& args, int tokens)
        : a(args), blocks(args.num_kv_heads * (kD / 8)) {
        const int64_t w = static_cast<int64_t>(blockIdx.x) * kSlotWarps + (threadIdx.x >> 5);
        is_v = (w & 1) != 0;
        token0 = (w >> 1) * tokens;
        const int64_t left = a.num_tokens - token0;
        total = static_cast<int>(left < tokens ? (left > 0 ? left : 0) : tokens) * blocks;
        inv = (65536u + blocks - 1) / blocks;
        shift = 31 - __clz(a.page_size);
        row0 = kOne && total > 0 ? row_of(a.slot_map[token0]) : -1;
    }
    // The token (from token0) of block u < 32 (u times inv's excess is below 2^16).
    __device__ __forceinline__ int token_of(int u) const {
        return kOne ? 0 : static_cast<int>((u * inv) >> 16);
    }
    // Pool row of a slot's head 0 (below 2^31); negative without a slot.
    __device__ __forceinline__ int32_t row_of(int32_t slot) const {
        if (slot < 0 || slot >= static_cast<int64_t>(a.num_pages) << shift) return -1;
        return (((slot >> shift) * a.num_kv_heads) << shift) + (slot & (a.page_size - 1));
    }
    __device__ __forceinline__ int32_t load_row(int t) const {
        return kOne ? row0 : row_of(a.slot_map[token0 + t]);
    }
    __device__ __forceinline__ int64_t head_row(int32_t row, int e) const {
        return row + ((e / (kD / 8)) << shift);
    }
};

template <int kKv, int kD, bool kOne>
__global__ void __launch_bounds__(kSlotThreads)
write_slots_kernel(const KvDst dst, const uint16_t* __restrict__ k_new,
                   const uint16_t* __restrict__ v_new, const SlotArgs a, int tokens) {
    launch_dependents();
    grid_dependency_wait();
    constexpr int kInFlight = kFlight<kOne>;
    const SlotWork<kD, kOne> w(a, tokens);
    if (kOne && w.row0 < 0) return;
    const int64_t stride = w.is_v ? a.v_stride : a.k_stride;
    const uint16_t* const src = (w.is_v ? v_new : k_new) + w.token0 * stride;
    void* const cache = w.is_v ? dst.v : dst.k;
    uint32_t* const params = w.is_v ? dst.v_params : dst.k_params;
    const float scale = w.is_v ? dst.v_scale : dst.k_scale;
    for (int u0 = threadIdx.x & 31; u0 < w.total; u0 += 32 * kInFlight) {
        uint4 raw[kInFlight];
        int32_t row[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, t = w.token_of(u);
            row[i] = u < w.total ? w.load_row(t) : -1;
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, t = w.token_of(u);
            if (u < w.total && row[i] >= 0)
                raw[i] = *reinterpret_cast<const uint4*>(src + t * stride + (u - t * w.blocks) * 8);
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, e = u - w.token_of(u) * w.blocks;
            if (u < w.total && row[i] >= 0)
                store8<kKv>(cache, params, w.head_row(row[i], e), kD, e % (kD / 8), raw[i], scale);
        }
    }
}

template <int kKv, int kD, bool kOne>
__global__ void __launch_bounds__(kSlotThreads)
read_slots_kernel(const KvDst src, uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                  const SlotArgs a, int tokens) {
    launch_dependents();
    grid_dependency_wait();
    constexpr int kInFlight = kFlight<kOne>;
    const SlotWork<kD, kOne> w(a, tokens);
    const int64_t stride = w.is_v ? a.v_stride : a.k_stride;
    uint16_t* const out = (w.is_v ? v_out : k_out) + w.token0 * stride;
    const void* const cache = w.is_v ? src.v : src.k;
    const uint32_t* const params = w.is_v ? src.v_params : src.k_params;
    const float scale = w.is_v ? src.v_scale : src.k_scale;
    for (int u0 = threadIdx.x & 31; u0 < w.total; u0 += 32 * kInFlight) {
        Held8 raw[kInFlight];
        int32_t row[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, t = w.token_of(u);
            row[i] = u < w.total ? w.load_row(t) : -1;
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, e = u - w.token_of(u) * w.blocks;
            if (row[i] >= 0)
                raw[i] = load8<kKv>(cache, params, w.head_row(row[i], e), kD, e % (kD / 8));
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int u = u0 + 32 * i, t = w.token_of(u);
            if (u < w.total)
                *reinterpret_cast<uint4*>(out + t * stride + (u - t * w.blocks) * 8) =
                    row[i] >= 0 ? decode8<kKv>(raw[i], scale) : make_uint4(0, 0, 0, 0);
        }
    }
}

static int slot_tokens(const SlotArgs& a) {
    const int blocks = a.num_kv_heads * (a.head_dim / 8);
    return blocks >= 32 ? 1 : 32 / blocks;
}

template <typename K, typename... A>
static cudaError_t launch_slots(K kernel, const SlotArgs& a, cudaStream_t stream, A... args) {
    const int tokens = slot_tokens(a);
    const int64_t warps = 2 * ((static_cast<int64_t>(a.num_tokens) - 1) / tokens + 1);
    PdlLaunch l(dim3(static_cast<unsigned>((warps - 1) / kSlotWarps + 1)), dim3(kSlotThreads), 0,
                stream);
    return cudaLaunchKernelEx(&l.cfg, kernel, args..., a, tokens);
}

#define PKV_SLOT_KERNEL(NAME, KV, D, ONE)                                                   \
    (ONE ? PKV_SLOT_KERNEL_(NAME, KV, D, true) : PKV_SLOT_KERNEL_(NAME, KV, D, false))
#define PKV_SLOT_KERNEL_(NAME, KV, D, ONE)                                                  \
    (KV == kKvFp8    ? (D == 64 ? NAME<kKvFp8, 64, ONE> : NAME<kKvFp8, 128, ONE>)             \
     : KV == kKvBf16 ? (D == 64 ? NAME<kKvBf16, 64, ONE> : NAME<kKvBf16, 128, ONE>)           \
                     : (D == 64 ? NAME<kKvInt4, 64, ONE> : NAME<kKvInt4, 128, ONE>))

cudaError_t launch_write_slots(const KvDst& dst, const uint16_t* k_new, const uint16_t* v_new,
                               const SlotArgs& a, cudaStream_t stream) {
    auto* kernel = PKV_SLOT_KERNEL(write_slots_kernel, dst.kv, a.head_dim, slot_tokens(a) == 1);
    return launch_slots(kernel, a, stream, dst, k_new, v_new);
}

cudaError_t launch_read_slots(const KvDst& src, uint16_t* k_out, uint16_t* v_out,
                              const SlotArgs& a, cudaStream_t stream) {
    auto* kernel = PKV_SLOT_KERNEL(read_slots_kernel, src.kv, a.head_dim, slot_tokens(a) == 1);
    return launch_slots(kernel, a, stream, src, k_out, v_out);
}

}  // namespace pkv
