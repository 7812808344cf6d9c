// e4m3 codes with one fp32 scale per block of 128: activations per token and 128 channels,
// weights per 128 x 128 block.
//
// a = max(max|x|, 2^-100), s = a/448, code = the e4m3 value nearest to x*448/a (exactly, halves to
// even). 448 is e4m3's largest magnitude, so the block's largest value lands on the top code; the
// floor keeps s and r = 448/a normal fp32 numbers for every input (an all-zero block gets s =
// 2^-100/448 and zero codes).
// max|x| is taken over integer magnitudes, which carries NaN and infinity along: such a block
// gets s = r = NaN and NaN codes.
//
// Both kernels read X once into registers and write its codes from there: bytes per value are
// the input's 2 or 4 plus 1, plus the scales. They are bound by HBM: 16384 x 11008 bf16 activations
// take 89 to 91 us (6.0 to 6.1 TB/s), fp32 146 us (6.2), 11008 x 4096 fp16 weights 24 us (5.6 TB/s; 22
// where the codes find room in L2), 4100 x 5136 fp32 weights 19 to 20 us (5.3 TB/s; 17 with one
// rounding and no bracket); a copy runs at 6.55 TB/s.
#include <algorithm>

#include "internal.cuh"
#include "vec.cuh"

namespace gq {

constexpr float kE4m3Max = 448.0f;

// a, s, and 448/a as r + r_lo
struct Fp8Scale {
    float a, s, r, r_lo;
};

__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t amax_bits) {
    const float a = amax_bits >= kInfBits ? __uint_as_float(0x7FC00000u)
                                          : fmaxf(__uint_as_float(amax_bits), 0x1p-100f);
    const float r = __fdiv_rn(kE4m3Max, a);
    return {a, __fdiv_rn(a, kE4m3Max), r, __fdiv_rn(fmaf(-r, a, kE4m3Max), a)};
}

// two products to two e4m3 codes, the first in the low byte (|x*r| <= 448 up to a rounding)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t o;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(o) : "f"(hi), "f"(lo));
    return o;
}

// The exact decision for four fp32 values, out of line: the fp64 quotient (never rounded onto a
// tie, from which it is at least 2^-30 of itself away) to fp32 with the last bit telling whether
// anything was cut off, to e4m3.
static __device__ __noinline__ uint32_t codes_exact(float4 v, float a) {
    float p[4];
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double q = static_cast<double>(x[i]) * 448.0 / static_cast<double>(a);
        const float f = __double2float_rz(q);
        p[i] = __uint_as_float(__float_as_uint(f) | (static_cast<double>(f) != q ? 1u : 0u));
    }
    return e4m3x2(p[0], p[1]) | (e4m3x2(p[2], p[3]) << 16);
}

// Four values' codes.
//   16-bit types: fma(v, r, v*r_lo) is the quotient within 2^-23 of itself, and the quotient itself
//   where that is an fp32 number; with v and a of 11 bits it is a tie or 2^-17 off one.
//   fp32: both ends of a bracket r (1 -+ 2^-22) (r and the products are within 2^-24) are rounded;
//   where their codes differ (one value in 200000, so four values in 50000, on normal data) the
//   exact decision is made.
template <typename T>
__device__ __forceinline__ uint32_t codes4(const float* v, const Fp8Scale& f) {
    float p[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = fmaf(v[i], f.r, v[i] * f.r_lo);
        return e4m3x2(p[0], p[1]) | (e4m3x2(p[2], p[3]) << 16);
    } else {
        const float up = f.r * (1.0f + 0x1p-22f), dn = f.r * (1.0f - 0x1p-22f);
        const uint32_t w = e4m3x2(v[0] * up, v[1] * up) | (e4m3x2(v[2] * up, v[3] * up) << 16);
        const uint32_t x = e4m3x2(v[0] * dn, v[1] * dn) | (e4m3x2(v[2] * dn, v[3] * dn) << 16);
        return w == x ? w : codes_exact(make_float4(v[0], v[1], v[2], v[3]), f.a);
    }
}

// one 16-byte vector's codes: 8 bytes (fp16, bf16) or 4 (fp32)
template <typename T>
__device__ __forceinline__ void store_codes_vec(uint8_t* p, const uint4& u, const Fp8Scale& f) {
    float v[Vec<T>::N];
    Vec<T>::unpack(u, v);
    if constexpr (Vec<T>::N == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(codes4<T>(v, f), codes4<T>(v + 4, f));
    else
        *reinterpret_cast<uint32_t*>(p) = codes4<T>(v, f);
}

// 16 values' codes, one 16-byte store
template <typename T>
__device__ __forceinline__ void store_codes16(uint8_t* p, const uint4* x, const Fp8Scale& f) {
    constexpr int N = Vec<T>::N;
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 16 / N; ++c) {
        float v[N];
        Vec<T>::unpack(x[c], v);
#pragma unroll
        for (int i = 0; i < N; i += 4) w[(c * N + i) / 4] = codes4<T>(v + i, f);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ uint32_t amax_vec(const uint4& u, uint32_t m) {
    float v[Vec<T>::N];
    Vec<T>::unpack(u, v);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) m = max(m, abs_bits(v[i]));
    return m;
}

// 32 bytes at once where they start on such a boundary, else as two halves.
__device__ __forceinline__ void load32(const void* p, int wide, uint4* x) {
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x[0].x), "=r"(x[0].y), "=r"(x[0].z), "=r"(x[0].w), "=r"(x[1].x),
                       "=r"(x[1].y), "=r"(x[1].z), "=r"(x[1].w)
                     : "l"(p));
    } else {
        x[0] = __ldcs(static_cast<const uint4*>(p));
        x[1] = __ldcs(static_cast<const uint4*>(p) + 1);
    }
}

// A CTA takes 8 tokens x 512 P channels. A warp takes one token: 8 lanes per 128-channel block, 16
// consecutive values per lane (one store of 16 codes), 4 blocks per pass, P passes, all loads
// first. The scales leave through shared memory as runs of 8 tokens. 16384 x 11008 bf16 takes 91 us
// with P = 4, 93 with 2, 119 with 1. Before the second multiply-add that makes the codes exact (6 us;
// two values per instruction 13) these were 82, 86 and 100, and 94 with P = 2 and a lane's two
// vectors 128 bytes apart (8-byte stores), 101 with 4 tokens x 128 channels per warp.
template <typename T, int P>
__global__ void __launch_bounds__(256) fp8_act_kernel(const T* __restrict__ X, int64_t n, int d,
                                                      uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales, int wide) {
    constexpr int N = Vec<T>::N, C = 16 / N;             // vectors of a lane and block
    __shared__ float sc[4 * P][8];
    pdl_wait();
    const int lane = lane_id(), part = lane & 7;
    const int nb = (d + 127) / 128;
    const int n_cb = (nb + 4 * P - 1) / (4 * P);
    const int64_t rb = blockIdx.x / n_cb;
    const int b0 = static_cast<int>(blockIdx.x - rb * n_cb) * 4 * P + (lane >> 3);
    const int64_t t = rb * 8 + warp_id();
    uint4 x[P][C];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int k = (b0 + 4 * p) * 128 + part * 16;    // d is a multiple of 16
#pragma unroll
        for (int c = 0; c < C; ++c) x[p][c] = make_uint4(0, 0, 0, 0);
        if (t < n && k < d) {
#pragma unroll
            for (int c = 0; c < C; c += 2) load32(X + t * d + k + c * N, wide, &x[p][c]);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) m = amax_vec<T>(x[p][c], m);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const Fp8Scale f = fp8_scale(m);
        const int k = (b0 + 4 * p) * 128 + part * 16;
        if (t < n && k < d) store_codes16<T>(codes + t * d + k, x[p], f);
        if (part == 0) sc[4 * p + (lane >> 3)][warp_id()] = f.s;
    }
    __syncthreads();
    if (threadIdx.x < 8 * 4 * P) {
        const int b = static_cast<int>(blockIdx.x - rb * n_cb) * 4 * P + (threadIdx.x >> 3);
        const int64_t row = rb * 8 + (threadIdx.x & 7);
        if (b < nb && row < n) scales[b * n + row] = sc[threadIdx.x >> 3][threadIdx.x & 7];
    }
}

// A CTA of 256 threads takes one 128 x 128 block, all of it in flight at once (32 KB of fp16): 8
// lanes per row, whose 16-byte vectors lie 8 apart, 4 rows per warp and step. Registers are bounded
// for three CTAs per SM with 16-bit inputs (with that, streaming loads and the overlapped launch
// 26.5 us became 21, codes in L2; with 32-byte loads as above 24).
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2)
    fp8_weight_kernel(const T* __restrict__ W, int d_out, int d_in, uint8_t* __restrict__ codes,
                      float* __restrict__ scales) {
    constexpr int N = Vec<T>::N, C = 16 / N;
    __shared__ uint32_t warp_max[8];
    pdl_wait();
    const int lane = lane_id(), part = lane & 7;
    const int nb = (d_in + 127) / 128;
    const int64_t rb = blockIdx.x / nb;
    const int b = static_cast<int>(blockIdx.x - rb * nb);
    uint4 x[4][C];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = rb * 128 + j * 32 + warp_id() * 4 + (lane >> 3);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = b * 128 + (c * 8 + part) * N;
            x[j][c] = make_uint4(0, 0, 0, 0);
            if (row < d_out && k < d_in)
                x[j][c] = __ldcs(reinterpret_cast<const uint4*>(W + row * d_in + k));
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int c = 0; c < C; ++c) m = amax_vec<T>(x[j][c], m);
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) warp_max[warp_id()] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, warp_max[w]);
    const Fp8Scale f = fp8_scale(m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = rb * 128 + j * 32 + warp_id() * 4 + (lane >> 3);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = b * 128 + (c * 8 + part) * N;
            if (row < d_out && k < d_in) store_codes_vec<T>(codes + row * d_in + k, x[j][c], f);
        }
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = f.s;
}

template <typename T, int P>
static gptq_status fp8_act_go(const void* X, int64_t n, int d, uint8_t* codes, float* scales,
                              int64_t ctas, cudaStream_t s) {
    if (ctas > 0x7FFFFFFF) return GPTQ_ERR_ARG;
    const int wide = (reinterpret_cast<uintptr_t>(X) & 31) == 0;
    GPTQ_CUDA_TRY(launch_pdl(fp8_act_kernel<T, P>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s,
                             static_cast<const T*>(X), n, d, codes, scales, wide));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

// Passes per CTA: 2 KB of a row at a time in 16 bits, 4 KB where that leaves 16 CTAs for every SM
// (16384 x 4096 fp16: 34.9 us, 35.7 with 2 KB; 2048 x 4096: 6.7 and 5.9), 1 KB where 2 KB leave fewer
// than 4 (513 x 5136: 2.6 us, 2.8 with 2 KB). In fp32 no more than 4 KB (16384 x 11008: 146 us, 156 with
// 8 KB).
template <typename T>
static gptq_status fp8_act_launch(const void* X, int64_t n, int d, uint8_t* codes, float* scales,
                                  cudaStream_t s) {
    auto ctas = [&](int p) { return ((n + 7) / 8) * ((d + 512 * p - 1) / (512 * p)); };
    if (sizeof(T) == 2 && ctas(4) >= 16 * num_sms())
        return fp8_act_go<T, 4>(X, n, d, codes, scales, ctas(4), s);
    if (ctas(2) >= 4 * num_sms()) return fp8_act_go<T, 2>(X, n, d, codes, scales, ctas(2), s);
    return fp8_act_go<T, 1>(X, n, d, codes, scales, ctas(1), s);
}

template <typename T>
static gptq_status fp8_weight_launch(const void* W, int d_out, int d_in, uint8_t* codes,
                                     float* scales, cudaStream_t s) {
    // at most 2^24 row blocks x 512 column blocks
    const int64_t blocks = ((static_cast<int64_t>(d_out) + 127) / 128) * ((d_in + 127) / 128);
    if (blocks > 0x7FFFFFFF) return GPTQ_ERR_ARG;
    GPTQ_CUDA_TRY(launch_pdl(fp8_weight_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                             s, static_cast<const T*>(W), d_out, d_in, codes, scales));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

static bool fp8_dtype_ok(int t) {
    return t == GPTQ_DTYPE_F16 || t == GPTQ_DTYPE_F32 || t == GPTQ_DTYPE_BF16;
}
static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Other CTAs read the input while one writes its codes and scales, so these may not share memory.
static bool fp8_apart(const void* x, int dtype, int64_t values, const void* codes,
                      const void* scales, int64_t n_scales) {
    const int64_t x_bytes = range_bytes(values, dtype == GPTQ_DTYPE_F32 ? 4 : 2);
    return !overlap(x, x_bytes, codes, values) && !overlap(x, x_bytes, scales, 4 * n_scales) &&
           !overlap(codes, values, scales, 4 * n_scales);
}

}  // namespace gq

extern "C" {

gptq_status fp8_quantize_act(const void* X, int x_dtype, int64_t n_tokens, int d, uint8_t* codes,
                             float* scales, void* stream) {
    if (!gq::fp8_dtype_ok(x_dtype) || n_tokens < 0 || n_tokens >= (int64_t(1) << 31))
        return GPTQ_ERR_ARG;
    if (d < 16 || d % 16 || d > 65536) return GPTQ_ERR_ARG;
    if (n_tokens == 0) return GPTQ_OK;
    if (!X || !codes || !scales || !gq::al16(X) || !gq::al16(codes) || !gq::al4(scales))
        return GPTQ_ERR_ARG;
    if (!gq::fp8_apart(X, x_dtype, n_tokens * d, codes, scales, n_tokens * ((d + 127) / 128)))
        return GPTQ_ERR_ARG;
    GPTQ_TRY(gq::check_device());
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (x_dtype) {
        case GPTQ_DTYPE_F16: return gq::fp8_act_launch<__half>(X, n_tokens, d, codes, scales, s);
        case GPTQ_DTYPE_BF16: return gq::fp8_act_launch<__nv_bfloat16>(X, n_tokens, d, codes, scales, s);
        default: return gq::fp8_act_launch<float>(X, n_tokens, d, codes, scales, s);
    }
}

gptq_status fp8_quantize_weight(const void* W, int w_dtype, int d_out, int d_in, uint8_t* codes,
                                float* scales, void* stream) {
    if (!W || !codes || !scales || !gq::fp8_dtype_ok(w_dtype)) return GPTQ_ERR_ARG;
    if (d_out < 1 || d_in < 16 || d_in % 16 || d_in > 65536) return GPTQ_ERR_ARG;
    if (!gq::al16(W) || !gq::al16(codes) || !gq::al4(scales)) return GPTQ_ERR_ARG;
    if (!gq::fp8_apart(W, w_dtype, static_cast<int64_t>(d_out) * d_in, codes, scales,
                       ((static_cast<int64_t>(d_out) + 127) / 128) * ((d_in + 127) / 128)))
        return GPTQ_ERR_ARG;
    GPTQ_TRY(gq::check_device());
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (w_dtype) {
        case GPTQ_DTYPE_F16: return gq::fp8_weight_launch<__half>(W, d_out, d_in, codes, scales, s);
        case GPTQ_DTYPE_BF16: return gq::fp8_weight_launch<__nv_bfloat16>(W, d_out, d_in, codes, scales, s);
        default: return gq::fp8_weight_launch<float>(W, d_out, d_in, codes, scales, s);
    }
}

}  // extern "C"
