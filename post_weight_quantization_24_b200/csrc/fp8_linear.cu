// Y = Xhat * What^T (+ R) from e4m3 codes with one scale per token and 128 channels (X) and per
// 128 x 128 block (W), on the 5th-generation tensor cores:
//   Y[t][o] = sum_b sx[b][t] * sw[o/128][b] * (sum_{c in block b} X8[t][c] * W8[o][c]) + R[t][o].
//
// The scales change every 128 channels, so the tensor cores sum one block at a time from zero
// (4 x tcgen05.mma kind::f8f6f4 of K = 32, fp32 accumulator in TMEM) and the sum over blocks
// is kept in registers: acc = fma(partial, sx*sw, acc), rounded to nearest.
//
// Persistent kernel, one CTA per SM, tiles of 128 tokens x 128 channels, ring of 6 stages:
//   warp 0     TMA producer: per block the 128 x 128-byte tiles of X and W (128-byte swizzle);
//   warp 1     TMEM allocator and MMA issuer, into one of four 128-column accumulators;
//   warps 2-9  promotion: a thread owns one token row and 64 columns.
// Tokens and channels past the edges are zero-filled by TMA and not stored.
// Every mbarrier wait is bounded; on timeout the kernel records GPTQ_ERR_TIMEOUT, drains its
// copies and MMAs, frees TMEM and returns.
#include <algorithm>

#include "internal.cuh"
#include "vec.cuh"

namespace gq {

namespace f8 {
constexpr int BM = 128, BN = 128, BK = 128, STAGES = 6;
constexpr int A_BYTES = BM * BK, B_BYTES = BN * BK;
constexpr int STAGE = A_BYTES + B_BYTES;
constexpr int ACCS = 4;                              // TMEM accumulators of BN columns
constexpr uint32_t TMEM_COLS = ACCS * BN;
constexpr int EPI_WARPS = 8, EPI_COLS = 64;          // 4 lane quarters x 2 column halves
constexpr int THREADS = (2 + EPI_WARPS) * 32;
constexpr int SMEM = 1024 + STAGES * STAGE + 256;
constexpr int BAND = 8;
constexpr uint32_t IDESC = umma_idesc_e4m3(BM, BN);
static_assert(SMEM <= 227 * 1024, "shared memory");
}  // namespace f8

struct F8Params {
    int n_tok, d_in, d_out;
    int n_mt, n_nt, n_kb;
    long long n_tiles;
    const float* sx;      // [n_kb x n_tok]
    const float* sw;      // [ceil(d_out/128) x n_kb]
    const void* R;
    void* Y;
    int vec_ok;           // rows of Y and R start on 16-byte boundaries
    int* status;
};

// Tiles run in bands of 8 token tiles with the token tile varying fastest, so the CTAs that run
// together share weight tiles and activation rows in L2.
__device__ __forceinline__ void f8_tile(const F8Params& p, long long t, int& m0, int& n0) {
    const long long per_band = static_cast<long long>(f8::BAND) * p.n_nt;
    const int band = static_cast<int>(t / per_band);
    const int rem = static_cast<int>(t - band * per_band);
    const int band_m = min(f8::BAND, p.n_mt - band * f8::BAND);
    m0 = (band * f8::BAND + rem % band_m) * f8::BM;
    n0 = (rem / band_m) * f8::BN;
}

// NC accumulated columns of one row -> Y (+ R), columns col0 .. min(col0 + NC, d_out)
template <typename T, int NC>
__device__ __forceinline__ void f8_store(const F8Params& p, int row, int col0, const float* acc) {
    constexpr int N = Vec<T>::N;
    if (row >= p.n_tok || col0 >= p.d_out) return;
    const int64_t off = static_cast<int64_t>(row) * p.d_out + col0;
    T* y = static_cast<T*>(p.Y) + off;
    const T* r = p.R ? static_cast<const T*>(p.R) + off : nullptr;
    const int left = p.d_out - col0;
    if (p.vec_ok) {       // d_out is a multiple of N
#pragma unroll
        for (int c = 0; c < NC; c += N) {
            if (c >= left) break;
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = acc[c + e];
            if (r) {
                float f[N];
                Vec<T>::unpack(*reinterpret_cast<const uint4*>(r + c), f);
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += f[e];
            }
            *reinterpret_cast<uint4*>(y + c) = Vec<T>::pack(v);
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if (c < left)
                y[c] = Vec<T>::from_float(acc[c] + (r ? Vec<T>::to_float(r[c]) : 0.0f));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(f8::THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                    const F8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + f8::STAGES * f8::STAGE);
    uint64_t* empty = full + f8::STAGES;
    uint64_t* acc_full = empty + f8::STAGES;
    uint64_t* acc_empty = acc_full + f8::ACCS;
    uint64_t* drained = acc_empty + f8::ACCS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < f8::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < f8::ACCS; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], f8::EPI_WARPS);
        }
        mbar_init(drained, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&wmap);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, f8::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (long long t = blockIdx.x; t < p.n_tiles && !*abort_flag; t += gridDim.x) {
                int m0, n0;
                f8_tile(p, t, m0, n0);
                for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                    const int st = it % f8::STAGES;
                    if (!mbar_wait(&empty[st], ((it / f8::STAGES) & 1) ^ 1)) {
                        set_status(p.status, GPTQ_ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t* sa = smem + st * f8::STAGE;
                    mbar_arrive_expect_tx(&full[st], f8::STAGE);
                    tma_load_2d(sa, &xmap, &full[st], kb * f8::BK, m0);
                    tma_load_2d(sa + f8::A_BYTES, &wmap, &full[st], kb * f8::BK, n0);
                }
            }
            const int n_tail = it < f8::STAGES ? it : f8::STAGES;
            for (int k = it - n_tail; k < it; ++k) {
                if (!mbar_wait(&full[k % f8::STAGES], (k / f8::STAGES) & 1)) {
                    set_status(p.status, GPTQ_ERR_TIMEOUT);
                    *abort_flag = 1;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (long long t = blockIdx.x; ok && t < p.n_tiles && !*abort_flag; t += gridDim.x) {
                for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                    const int st = it % f8::STAGES, b = it % f8::ACCS;
                    if (!mbar_wait(&acc_empty[b], ((it / f8::ACCS) & 1) ^ 1) ||
                        !mbar_wait(&full[st], (it / f8::STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * f8::BN);
                    const uint32_t s0 = smem_u32(smem + st * f8::STAGE);
#pragma unroll
                    for (int kk = 0; kk < f8::BK / 32; ++kk) {
                        // K-major rows of 128 B; a k-step of 32 codes is 32 B along the row
                        const uint64_t ad = umma_desc_sw128(s0 + kk * 32, 16, 1024);
                        const uint64_t bd = umma_desc_sw128(s0 + f8::A_BYTES + kk * 32, 16, 1024);
                        umma_f8(d_tmem, ad, bd, f8::IDESC, kk > 0 ? 1u : 0u);
                    }
                    umma_commit(&empty[st]);
                    umma_commit(&acc_full[b]);
                }
            }
            if (!ok) {
                set_status(p.status, GPTQ_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            umma_commit(drained);
            if (!mbar_wait(drained, 0)) set_status(p.status, GPTQ_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t t_lane = static_cast<uint32_t>(32 * q) << 16;
        int it = 0;
        bool stop = false;
        for (long long t = blockIdx.x; t < p.n_tiles && !stop; t += gridDim.x) {
            int m0, n0;
            f8_tile(p, t, m0, n0);
            const int row = m0 + 32 * q + lane;
            const float* sx = p.sx + min(row, p.n_tok - 1);
            const float* sw = p.sw + static_cast<int64_t>(n0 / 128) * p.n_kb;
            float acc[f8::EPI_COLS];
#pragma unroll
            for (int k = 0; k < f8::EPI_COLS; ++k) acc[k] = 0.0f;
            for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                const int b = it % f8::ACCS;
                const float f = __ldg(sx + static_cast<int64_t>(kb) * p.n_tok) * __ldg(sw + kb);
                int ok = 1;
                if (lane == 0) ok = mbar_wait(&acc_full[b], (it / f8::ACCS) & 1) ? 1 : 0;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok || __shfl_sync(0xffffffffu, *abort_flag, 0)) {
                    if (lane == 0 && !ok) {
                        set_status(p.status, GPTQ_ERR_TIMEOUT);
                        *abort_flag = 1;
                    }
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint32_t t_col = static_cast<uint32_t>(b * f8::BN + f8::EPI_COLS * half);
                uint32_t r[f8::EPI_COLS / 32][32];
#pragma unroll
                for (int j = 0; j < f8::EPI_COLS / 32; ++j)
                    tmem_ld_32x32b_x32(tmem_base + t_lane + t_col + 32 * j, r[j]);
                tmem_ld_wait_for(r[0]);
#pragma unroll
                for (int j = 1; j < f8::EPI_COLS / 32; ++j) tmem_ld_use(r[j]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
                for (int j = 0; j < f8::EPI_COLS / 32; ++j)
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        acc[32 * j + k] = fmaf(__uint_as_float(r[j][k]), f, acc[32 * j + k]);
            }
            if (!stop) f8_store<T, f8::EPI_COLS>(p, row, n0 + f8::EPI_COLS * half, acc);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, f8::TMEM_COLS);
}

template <typename T>
static gptq_status fp8_gemm_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                   cudaStream_t s) {
    GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, f8::SMEM));
    p.vec_ok = p.d_out % Vec<T>::N == 0;
    CUtensorMap xmap, wmap;
    GPTQ_TRY(encode_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(X8),
                                  p.d_in, p.n_tok, p.d_in, f8::BK, f8::BM,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    GPTQ_TRY(encode_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(W8),
                                  p.d_in, p.d_out, p.d_in, f8::BK, f8::BN,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    p.n_mt = (p.n_tok - 1) / f8::BM + 1;
    p.n_nt = (p.d_out - 1) / f8::BN + 1;
    p.n_tiles = static_cast<long long>(p.n_mt) * p.n_nt;
    const int grid = static_cast<int>(std::min<long long>(p.n_tiles, num_sms()));
    fp8_gemm_kernel<T><<<grid, f8::THREADS, f8::SMEM, s>>>(xmap, wmap, p);
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

}  // namespace gq

extern "C" gptq_status fp8_linear(const uint8_t* X8, const float* x_scales, int64_t n_tokens,
                                  int d_in, const uint8_t* W8, const float* w_scales, int d_out,
                                  const void* R, void* Y, int y_dtype, int* status_dev,
                                  void* stream) {
    if (n_tokens < 0 || n_tokens >= (int64_t(1) << 31)) return GPTQ_ERR_ARG;
    if (d_in < 16 || d_in % 16 || d_in > 65536 || d_out < 1) return GPTQ_ERR_ARG;
    if (y_dtype != GPTQ_DTYPE_F16 && y_dtype != GPTQ_DTYPE_F32 && y_dtype != GPTQ_DTYPE_BF16)
        return GPTQ_ERR_ARG;
    if (n_tokens == 0) return GPTQ_OK;
    auto al = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    if (!X8 || !x_scales || !W8 || !w_scales || !Y || !al(X8, 16) || !al(W8, 16) || !al(Y, 16) ||
        (R && !al(R, 16)) || !al(x_scales, 4) || !al(w_scales, 4) || !al(status_dev, 4))
        return GPTQ_ERR_ARG;
    GPTQ_TRY(gq::check_device());
    gq::F8Params p{};
    p.n_tok = static_cast<int>(n_tokens);
    p.d_in = d_in;
    p.d_out = d_out;
    p.n_kb = (d_in + 127) / 128;
    p.sx = x_scales;
    p.sw = w_scales;
    p.R = R;
    p.Y = Y;
    p.status = status_dev;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (y_dtype) {
        case GPTQ_DTYPE_F16: return gq::fp8_gemm_launch<__half>(X8, W8, p, s);
        case GPTQ_DTYPE_BF16: return gq::fp8_gemm_launch<__nv_bfloat16>(X8, W8, p, s);
        default: return gq::fp8_gemm_launch<float>(X8, W8, p, s);
    }
}
