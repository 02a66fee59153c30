// kv_slots.cu -- token writes into cache slots named by a slot map, and reads
// of such slots back as bf16, for FP8, BF16 and INT4 caches.
//
// One thread moves one 8-value block (16 bytes of bf16) of K and the same
// block of V, so two loads are in flight per thread and each 128-byte line of
// the token rows is read by 8 consecutive lanes; an INT4 group of 64 dims is
// exactly those 8 lanes, whose minimum and maximum meet in three shuffles.
#include "kv_codec.cuh"

namespace pkv {

constexpr int kSlotThreads = 256;

// Block of the calling thread: its token and the (head, 8-dim block) in the
// token's row.  The blocks of `tokens_per_cta` consecutive tokens form a CTA's
// work, kSlotThreads at a time (a row has a multiple of 8 blocks, so 8
// consecutive lanes always share token and head).
template <typename F>
__device__ __forceinline__ void for_each_block(const SlotArgs& a, int tokens_per_cta, F f) {
    const int row_blocks = a.num_kv_heads * (a.head_dim / 8);
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
    const int64_t left = a.num_tokens - t0;
    const int tokens = static_cast<int>(left < tokens_per_cta ? left : tokens_per_cta);
    const int total = tokens * row_blocks;
    const int64_t slots = static_cast<int64_t>(a.num_pages) * a.page_size;
    for (int e = threadIdx.x; e < total; e += kSlotThreads) {
        const int t = e / row_blocks;
        const int r = e - t * row_blocks;
        const int h = r / (a.head_dim / 8);
        const int d8 = r - h * (a.head_dim / 8);
        const int32_t slot = a.slot_map[t0 + t];
        int64_t row = -1;
        if (slot >= 0 && slot < slots) {
            const int32_t page = slot / a.page_size;
            row = (static_cast<int64_t>(page) * a.num_kv_heads + h) * a.page_size +
                  (slot - page * a.page_size);
        }
        f(t0 + t, static_cast<int64_t>(r) * 8, row, d8);
    }
}

template <int kKv>
__global__ void __launch_bounds__(kSlotThreads)
write_slots_kernel(const KvDst dst, const uint16_t* __restrict__ k_new,
                   const uint16_t* __restrict__ v_new, const SlotArgs a, int tokens_per_cta) {
    launch_dependents();
    grid_dependency_wait();
    for_each_block(a, tokens_per_cta, [&](int64_t t, int64_t off, int64_t row, int d8) {
        if (row < 0) return;
        const uint4 k = *reinterpret_cast<const uint4*>(k_new + t * a.k_stride + off);
        const uint4 v = *reinterpret_cast<const uint4*>(v_new + t * a.v_stride + off);
        store8<kKv>(dst.k, dst.k_params, row, a.head_dim, d8, k, dst.k_scale);
        store8<kKv>(dst.v, dst.v_params, row, a.head_dim, d8, v, dst.v_scale);
    });
}

template <int kKv>
__global__ void __launch_bounds__(kSlotThreads)
read_slots_kernel(const KvDst src, uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                  const SlotArgs a, int tokens_per_cta) {
    launch_dependents();
    grid_dependency_wait();
    for_each_block(a, tokens_per_cta, [&](int64_t t, int64_t off, int64_t row, int d8) {
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        if (row >= 0) {
            k = load8<kKv>(src.k, src.k_params, row, a.head_dim, d8, src.k_scale);
            v = load8<kKv>(src.v, src.v_params, row, a.head_dim, d8, src.v_scale);
        }
        *reinterpret_cast<uint4*>(k_out + t * a.k_stride + off) = k;
        *reinterpret_cast<uint4*>(v_out + t * a.v_stride + off) = v;
    });
}

// Tokens per CTA: one pass of the CTA's threads over its blocks, or one token
// where a row has more.
static int slot_tokens_per_cta(const SlotArgs& a) {
    const int row_blocks = a.num_kv_heads * (a.head_dim / 8);
    const int n = kSlotThreads / row_blocks;
    return n < 1 ? 1 : n;
}

cudaError_t launch_write_slots(const KvDst& dst, const uint16_t* k_new, const uint16_t* v_new,
                               const SlotArgs& a, cudaStream_t stream) {
    const int per = slot_tokens_per_cta(a);
    PdlLaunch l(dim3(static_cast<unsigned>((a.num_tokens - 1) / per + 1)), dim3(kSlotThreads), 0,
                stream);
    auto* kernel = dst.kv == kKvFp8    ? write_slots_kernel<kKvFp8>
                   : dst.kv == kKvBf16 ? write_slots_kernel<kKvBf16>
                                       : write_slots_kernel<kKvInt4>;
    return cudaLaunchKernelEx(&l.cfg, kernel, dst, k_new, v_new, a, per);
}

cudaError_t launch_read_slots(const KvDst& src, uint16_t* k_out, uint16_t* v_out,
                              const SlotArgs& a, cudaStream_t stream) {
    const int per = slot_tokens_per_cta(a);
    PdlLaunch l(dim3(static_cast<unsigned>((a.num_tokens - 1) / per + 1)), dim3(kSlotThreads), 0,
                stream);
    auto* kernel = src.kv == kKvFp8    ? read_slots_kernel<kKvFp8>
                   : src.kv == kKvBf16 ? read_slots_kernel<kKvBf16>
                                       : read_slots_kernel<kKvInt4>;
    return cudaLaunchKernelEx(&l.cfg, kernel, src, k_out, v_out, a, per);
}

}  // namespace pkv
