// The quantised key/value cache: keys and values get the group min-max quantizer of quant.cuh
// (per token and head, groups along head_dim) as they are written into a paged cache, and are
// read back as scale * (code - zero).
//
// Both kernels move each byte once and are bound by HBM (long calls) or by launch latency
// (a decode step's few tokens). A token's heads lie together in the cache, so its
// n_heads * head_dim elements are one contiguous row in every array, and the kernels see rows
// of `width` elements in chunks of 8; a group is 2 to 32 consecutive chunks of one row.
#include <algorithm>

#include "internal.cuh"
#include "quant.cuh"
#include "vec.cuh"

namespace gq {

struct KvParams {
    int64_t n_slots;       // slots of one plane (keys; the values' plane follows)
    int width, wc;         // elements and 8-element chunks of a token's row
    int ng;                // groups of a row
    int tpg;               // chunks per group: 2, 4, 8, 16 or 32
    uint8_t* codes;
    uint16_t* scales;
    uint16_t* zeros;
    int* status;
};

template <typename T>
__device__ __forceinline__ void kv_load8(const T* p, float* v) {
    Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), v);
    if constexpr (Vec<T>::N == 4) Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p) + 1), v + 4);
}

template <typename T>
__device__ __forceinline__ void kv_store8(T* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = Vec<T>::pack(v);
    if constexpr (Vec<T>::N == 4) *(reinterpret_cast<uint4*>(p) + 1) = Vec<T>::pack(v + 4);
}

constexpr uint16_t kHalfNan = 0x7E00;

// A thread takes one chunk of 8 elements; the chunks of a token (keys, then values) run over
// threadIdx.x, tokens over threadIdx.y and the grid. The tpg lanes of a group reduce its range
// with shuffles, and each computes the group's scalars (fp64, quant.cuh) for its own chunk.
template <typename T, int BITS>
__global__ void __launch_bounds__(256) kv_write_kernel(const T* __restrict__ K,
                                                       const T* __restrict__ V, int64_t n,
                                                       int64_t k_stride, int64_t v_stride,
                                                       const int64_t* __restrict__ slots,
                                                       const KvParams p) {
    constexpr int MAXQ = (1 << BITS) - 1;
    const int chunks = 2 * p.wc;
    const int64_t t_step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    // every lane takes every iteration (full-mask shuffles); lanes without work hold zeros
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * blockDim.y; t0 < n; t0 += t_step) {
        const int64_t t = t0 + threadIdx.y;
        int64_t slot = -1;
        if (t < n) slot = slots[t];
        if (slot >= p.n_slots) {
            if (threadIdx.x == 0) set_status(p.status, GPTQ_ERR_ARG);
            slot = -1;
        }
        for (int c0 = 0; c0 < chunks; c0 += blockDim.x) {
            const int c = c0 + threadIdx.x;
            const bool ok = slot >= 0 && c < chunks;
            const int plane = c >= p.wc ? 1 : 0;
            const int wc = c - plane * p.wc;              // chunk of the row
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (ok) kv_load8(plane ? V + t * v_stride + 8 * wc : K + t * k_stride + 8 * wc, v);
            float mn = v[0], mx = v[0];
            uint32_t am = abs_bits(v[0]);
#pragma unroll
            for (int i = 1; i < 8; ++i) {
                mn = fminf(mn, v[i]);
                mx = fmaxf(mx, v[i]);
                am = max(am, abs_bits(v[i]));
            }
            for (int o = p.tpg / 2; o > 0; o >>= 1) {
                mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
            }
            if (!ok) continue;
            uint16_t sb = kHalfNan, zb = 0;
            int q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (am < kInfBits) {
                const QParams g = group_params(mn, mx, MAXQ);
                if (g.scale <= 65504.0f) {
                    sb = half_bits(g.scale);
                    zb = half_bits(g.zero);
#pragma unroll
                    for (int i = 0; i < 8; ++i) q[i] = quant_code(v[i], g, MAXQ);
                }
            }
            const int64_t row = plane * p.n_slots + slot;
            if (BITS == 4) {
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) w |= static_cast<uint32_t>(q[i]) << (4 * i);
                *reinterpret_cast<uint32_t*>(p.codes + (row * p.wc + wc) * 4) = w;
            } else {
                uint2 w;
                w.x = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
                w.y = q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24);
                *reinterpret_cast<uint2*>(p.codes + (row * p.wc + wc) * 8) = w;
            }
            if ((wc & (p.tpg - 1)) == 0) {
                const int64_t gi = row * p.ng + wc / p.tpg;
                p.scales[gi] = sb;
                p.zeros[gi] = zb;
            }
        }
    }
}

// The sequence of row t: the largest b with cu[b] <= t, by a 32-way search of the warp (-1 when
// t < cu[0]).
__device__ __forceinline__ int kv_find_seq(const int32_t* __restrict__ cu, int n_seqs, int64_t t) {
    int lo = 0, count = n_seqs + 1;               // cu[lo .. lo + count) holds the answer
    while (count > 0) {
        const int step = (count + 31) / 32;
        const int i = lo + lane_id() * step;
        const bool below = lane_id() * step < count && __ldg(cu + i) <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, below));
        if (k == 0) return lo - 1;                // only in the first round, or none further on
        const int end = lo + count;
        lo += (k - 1) * step;
        if (step == 1) return lo;
        // cu[lo] <= t: look among the entries behind it, up to the next probe
        ++lo;
        count = min(step - 1, end - lo);
    }
    return lo - 1;
}

// A warp takes one row of the output (a token's keys and values); lanes run over its chunks.
template <typename T, int BITS>
__global__ void __launch_bounds__(256) kv_read_kernel(const KvParams p, int page_size,
                                                      int64_t n_pages,
                                                      const int32_t* __restrict__ table,
                                                      int n_seqs, int max_pages,
                                                      const int32_t* __restrict__ cu,
                                                      int64_t total, T* __restrict__ K,
                                                      T* __restrict__ V) {
    const int lane = lane_id(), chunks = 2 * p.wc;
    const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp_id(); t < total; t += step) {
        const int b = kv_find_seq(cu, n_seqs, t);
        if (b < 0 || b >= n_seqs) continue;       // a row of no sequence: left as it was
        const int64_t pos = t - __ldg(cu + b);
        const int64_t pi = pos / page_size;
        int64_t page = -1;
        if (pos >= 0 && pi < max_pages) page = __ldg(table + static_cast<int64_t>(b) * max_pages + pi);
        const bool found = page >= 0 && page < n_pages;
        if (!found && lane == 0) set_status(p.status, GPTQ_ERR_ARG);
        const int64_t slot = page * page_size + (pos - pi * page_size);
#pragma unroll 4
        for (int c = lane; c < chunks; c += 32) {
            const int plane = c >= p.wc ? 1 : 0;
            const int wc = c - plane * p.wc;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (found) {
                const int64_t row = plane * p.n_slots + slot;
                const int64_t gi = row * p.ng + wc / p.tpg;
                const float s = __half2float(__ushort_as_half(__ldg(p.scales + gi)));
                const float z = __half2float(__ushort_as_half(__ldg(p.zeros + gi)));
                if (BITS == 4) {
                    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p.codes) + row * p.wc + wc);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = s * (static_cast<float>((w >> (4 * i)) & 15u) - z);
                } else {
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.codes) + row * p.wc + wc);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = s * (static_cast<float>((w.x >> (8 * i)) & 255u) - z);
                        v[4 + i] = s * (static_cast<float>((w.y >> (8 * i)) & 255u) - z);
                    }
                }
            }
            kv_store8((plane ? V : K) + t * p.width + 8 * wc, v);
        }
    }
}

template <typename T>
static gptq_status kv_write_launch(const void* K, const void* V, int64_t n, int64_t ks, int64_t vs,
                                   const int64_t* slots, int bits, const KvParams& p,
                                   cudaStream_t s) {
    int bx = 32;
    while (bx < 2 * p.wc && bx < 256) bx *= 2;
    const dim3 block(bx, 256 / bx);
    const int64_t want = (n + block.y - 1) / block.y;
    const int grid = static_cast<int>(std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * 64));
    const T* k = static_cast<const T*>(K);
    const T* v = static_cast<const T*>(V);
    if (bits == 4)
        kv_write_kernel<T, 4><<<grid, block, 0, s>>>(k, v, n, ks, vs, slots, p);
    else
        kv_write_kernel<T, 8><<<grid, block, 0, s>>>(k, v, n, ks, vs, slots, p);
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

template <typename T>
static gptq_status kv_read_launch(const KvParams& p, int page_size, int64_t n_pages,
                                  const int32_t* table, int n_seqs, int max_pages,
                                  const int32_t* cu, int64_t total, void* K, void* V, int bits,
                                  cudaStream_t s) {
    const int64_t want = (total + 7) / 8;
    const int grid = static_cast<int>(std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * 64));
    T* k = static_cast<T*>(K);
    T* v = static_cast<T*>(V);
    if (bits == 4)
        kv_read_kernel<T, 4><<<grid, 256, 0, s>>>(p, page_size, n_pages, table, n_seqs, max_pages,
                                                  cu, total, k, v);
    else
        kv_read_kernel<T, 8><<<grid, 256, 0, s>>>(p, page_size, n_pages, table, n_seqs, max_pages,
                                                  cu, total, k, v);
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

static bool kv_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// the checks and the row geometry that writing and reading share
static gptq_status kv_params(int dtype, int n_heads, int head_dim, int bits, int group_size,
                             int64_t n_slots, const void* codes, const void* scales,
                             const void* zeros, int* status, KvParams* p) {
    if (dtype != GPTQ_DTYPE_F16 && dtype != GPTQ_DTYPE_F32 && dtype != GPTQ_DTYPE_BF16)
        return GPTQ_ERR_ARG;
    if (bits != 4 && bits != 8) return GPTQ_ERR_ARG;
    if (group_size < 16 || group_size > 256 || (group_size & (group_size - 1))) return GPTQ_ERR_ARG;
    if (n_heads < 1 || head_dim < 16 || head_dim > 65536 || head_dim % group_size ||
        static_cast<int64_t>(n_heads) * head_dim > 65536)
        return GPTQ_ERR_ARG;
    if (n_slots < 1 || n_slots > (int64_t(1) << 40)) return GPTQ_ERR_ARG;
    if (!codes || !scales || !zeros || !kv_aligned(codes, 16) || !kv_aligned(scales, 2) ||
        !kv_aligned(zeros, 2) || !kv_aligned(status, 4))
        return GPTQ_ERR_ARG;
    p->n_slots = n_slots;
    p->width = n_heads * head_dim;
    p->wc = p->width / 8;
    p->ng = p->width / group_size;
    p->tpg = group_size / 8;
    p->codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    p->scales = static_cast<uint16_t*>(const_cast<void*>(scales));
    p->zeros = static_cast<uint16_t*>(const_cast<void*>(zeros));
    p->status = status;
    return GPTQ_OK;
}

}  // namespace gq

extern "C" {

gptq_status kv_cache_write(const void* K, const void* V, int dtype, int64_t n_tokens,
                           int64_t k_stride, int64_t v_stride, int n_heads, int head_dim,
                           const int64_t* slots, int64_t n_slots, int bits, int group_size,
                           uint8_t* codes, uint16_t* scales, uint16_t* zeros, int* status_dev,
                           void* stream) {
    gq::KvParams p;
    GPTQ_TRY(gq::kv_params(dtype, n_heads, head_dim, bits, group_size, n_slots, codes, scales, zeros,
                           status_dev, &p));
    if (n_tokens < 0 || n_tokens >= (int64_t(1) << 31)) return GPTQ_ERR_ARG;
    const int vec = dtype == GPTQ_DTYPE_F32 ? 4 : 8;
    if (k_stride < 0 || v_stride < 0 || k_stride % vec || v_stride % vec ||
        k_stride > (int64_t(1) << 31) || v_stride > (int64_t(1) << 31))
        return GPTQ_ERR_ARG;
    if (n_tokens == 0) return GPTQ_OK;
    if (!K || !V || !slots || !gq::kv_aligned(K, 16) || !gq::kv_aligned(V, 16) ||
        !gq::kv_aligned(slots, 8))
        return GPTQ_ERR_ARG;
    GPTQ_TRY(gq::check_device());
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case GPTQ_DTYPE_F16:
            return gq::kv_write_launch<__half>(K, V, n_tokens, k_stride, v_stride, slots, bits, p, s);
        case GPTQ_DTYPE_BF16:
            return gq::kv_write_launch<__nv_bfloat16>(K, V, n_tokens, k_stride, v_stride, slots, bits,
                                                      p, s);
        default:
            return gq::kv_write_launch<float>(K, V, n_tokens, k_stride, v_stride, slots, bits, p, s);
    }
}

gptq_status kv_cache_read(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros,
                          int64_t n_pages, int page_size, int n_heads, int head_dim, int bits,
                          int group_size, const int32_t* page_table, int n_seqs, int max_pages,
                          const int32_t* cu_lens, int64_t total, void* K, void* V, int dtype,
                          int* status_dev, void* stream) {
    if (n_pages < 1 || n_pages > 0x7FFFFFFF || page_size < 1) return GPTQ_ERR_ARG;
    gq::KvParams p;
    GPTQ_TRY(gq::kv_params(dtype, n_heads, head_dim, bits, group_size, n_pages * page_size, codes,
                           scales, zeros, status_dev, &p));
    if (n_seqs < 0 || n_seqs > (1 << 30) || max_pages < 0 || total < 0 ||
        total >= (int64_t(1) << 31))
        return GPTQ_ERR_ARG;
    if (total == 0 || n_seqs == 0) return GPTQ_OK;
    if ((!page_table && max_pages) || !cu_lens || !K || !V || !gq::kv_aligned(page_table, 4) ||
        !gq::kv_aligned(cu_lens, 4) || !gq::kv_aligned(K, 16) || !gq::kv_aligned(V, 16))
        return GPTQ_ERR_ARG;
    GPTQ_TRY(gq::check_device());
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case GPTQ_DTYPE_F16:
            return gq::kv_read_launch<__half>(p, page_size, n_pages, page_table, n_seqs, max_pages,
                                              cu_lens, total, K, V, bits, s);
        case GPTQ_DTYPE_BF16:
            return gq::kv_read_launch<__nv_bfloat16>(p, page_size, n_pages, page_table, n_seqs,
                                                     max_pages, cu_lens, total, K, V, bits, s);
        default:
            return gq::kv_read_launch<float>(p, page_size, n_pages, page_table, n_seqs, max_pages,
                                             cu_lens, total, K, V, bits, s);
    }
}

}  // extern "C"
