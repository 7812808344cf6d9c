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
    int n_tiles;
    const float* sx;      // [n_kb x n_tok]
    const float* sw;      // [ceil(d_out/128) x n_kb]
    const void* R;
    void* Y;
    int vec_ok;           // rows of Y and R start on 16-byte boundaries
    int* status;
};

// Tiles run in bands of 8 token tiles with the token tile varying fastest, so the CTAs that run
// together share weight tiles and activation rows in L2.
__device__ __forceinline__ void f8_tile(const F8Params& p, int t, int bm, int bn, int& m0,
                                        int& n0) {
    const int per_band = f8::BAND * p.n_nt;
    const int band = t / per_band;
    const int rem = t - band * per_band;
    const int band_m = min(f8::BAND, p.n_mt - band * f8::BAND);
    m0 = (band * f8::BAND + rem % band_m) * bm;
    n0 = (rem / band_m) * bn;
}

// NC accumulated columns of one row -> Y (+ R), columns col0 .. min(col0 + NC, d_out)
template <typename T, int NC>
__device__ __forceinline__ void f8_store(const F8Params& p, int row, int col0,
                                         const uint64_t (&acc)[NC / 2]) {
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
            for (int e = 0; e < N; ++e) v[e] = f32x2_get(acc[(c + e) / 2], e & 1);
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
                y[c] = Vec<T>::from_float(f32x2_get(acc[c / 2], c & 1) +
                                          (r ? Vec<T>::to_float(r[c]) : 0.0f));
        }
    }
}

// acc += f * (NC/2 pairs of partial sums)
template <int NC>
__device__ __forceinline__ void f8_promote(uint64_t* acc, const uint32_t (&r)[NC], uint64_t f) {
#pragma unroll
    for (int k = 0; k < NC / 2; ++k) fma_f32x2(acc[k], f32x2(r[2 * k], r[2 * k + 1]), f);
}

// Wait of a whole warp, every lane on the barrier itself: true if it completed, else the timeout
// is recorded.
__device__ __forceinline__ bool f8_warp_wait(uint64_t* bar, uint32_t parity, int* status,
                                             volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity))) return true;
    set_status(status, GPTQ_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
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
            for (int t = blockIdx.x; t < p.n_tiles && !*abort_flag; t += gridDim.x) {
                int m0, n0;
                f8_tile(p, t, f8::BM, f8::BN, m0, n0);
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
            for (int t = blockIdx.x; ok && t < p.n_tiles && !*abort_flag; t += gridDim.x) {
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
        for (int t = blockIdx.x; t < p.n_tiles && !stop; t += gridDim.x) {
            int m0, n0;
            f8_tile(p, t, f8::BM, f8::BN, m0, n0);
            const int row = m0 + 32 * q + lane;
            const float* sx = p.sx + min(row, p.n_tok - 1);
            const float* sw = p.sw + static_cast<int64_t>(n0 / 128) * p.n_kb;
            uint64_t acc[f8::EPI_COLS / 2];
#pragma unroll
            for (int k = 0; k < f8::EPI_COLS / 2; ++k) acc[k] = 0;
            float sx_next = __ldg(sx), sw_next = __ldg(sw);
            for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                const int b = it % f8::ACCS;
                const uint32_t f = __float_as_uint(sx_next * sw_next);
                if (kb + 1 < p.n_kb) {
                    sx_next = __ldg(sx + static_cast<int64_t>(kb + 1) * p.n_tok);
                    sw_next = __ldg(sw + kb + 1);
                }
                if (!f8_warp_wait(&acc_full[b], (it / f8::ACCS) & 1, p.status, abort_flag)) {
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
                if (lane == 0) mbar_arrive_relaxed(&acc_empty[b]);
#pragma unroll
                for (int j = 0; j < f8::EPI_COLS / 32; ++j) f8_promote<32>(acc + 16 * j, r[j], f32x2(f, f));
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

static gptq_status f8_tiles(F8Params& p) {
    // tile numbers (with a launch's stride added) stay within 31 bits
    const long long n = static_cast<long long>(p.n_mt) * p.n_nt;
    if (n > 0x7FFF0000 || f8::BAND * static_cast<long long>(p.n_nt) > 0x7FFF0000) return GPTQ_ERR_ARG;
    p.n_tiles = static_cast<int>(n);
    return GPTQ_OK;
}

template <typename T>
static gptq_status fp8_gemm_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                   cudaStream_t s) {
    GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_gemm_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, f8::SMEM));
    CUtensorMap xmap, wmap;
    GPTQ_TRY(encode_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(X8),
                                  p.d_in, p.n_tok, p.d_in, f8::BK, f8::BM,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    GPTQ_TRY(encode_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(W8),
                                  p.d_in, p.d_out, p.d_in, f8::BK, f8::BN,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    p.n_mt = (p.n_tok - 1) / f8::BM + 1;
    p.n_nt = (p.d_out - 1) / f8::BN + 1;
    GPTQ_TRY(f8_tiles(p));
    const int grid = std::min(p.n_tiles, num_sms());
    fp8_gemm_kernel<T><<<grid, f8::THREADS, f8::SMEM, s>>>(xmap, wmap, p);
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

// ---------------------------------------------------------------------------------------
// Pair kernel for large calls: two CTAs of a cluster share one 256 x 256 tile (tcgen05
// cta_group::2). Each CTA loads its 128 tokens and half of the tile's channels per block, 32 KB
// for 8.4 M products instead of the 64 KB that four 128 x 128 tiles need, and promotes its own 128
// tokens x 256 channels. Synchronisation as in the Hessian's pair kernel: both CTAs' bytes
// complete on the leader's stage barrier, the leader's commits arrive on both CTAs' barriers, both
// CTAs' promotion warps release an accumulator on the leader's.
//
// Two issuer warps take the blocks in turn, each with its own 256-column accumulator: a thread
// that commits and then waits on a barrier loses about 45 + 50 cycles per commit and wait, because
// nothing of its next block is queued meanwhile. One issuer took 648 cycles per block, two take
// the tensor pipe's 512 (measured on synthetic blocks; splitting N instead of the blocks took
// 692). Each of the two promotion warpgroups owns half of the columns.
// ---------------------------------------------------------------------------------------
namespace f8p {
constexpr int PT = 256;                              // pair tile edge
constexpr int BM = 128, BNC = 128;                   // tokens, channels loaded per CTA
constexpr int BK = 128, STAGES = 4;
constexpr int A_BYTES = BM * BK, STAGE = A_BYTES + BNC * BK;
constexpr int HN = 128;                              // columns of a promotion warpgroup
// Warpgroup 0 holds the producer and the two issuers, warpgroups 1 and 2 promote: a
// thread keeps one token's 128 sums and two 32-column loads in flight, more than an even share
// of registers.
constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int EPI_THREADS = EPI_WARPS * 32;
constexpr int THREADS = EPI_WARP0 * 32 + EPI_THREADS;
constexpr int REGS = 168, REGS_IO = 56, REGS_EPI = 224;
static_assert(REGS_IO * 128 + REGS_EPI * 256 <= REGS * THREADS, "register shares");
// A warp's rows leave through shared memory: boxes of 32 rows x 128 bytes (128-byte swizzle), two at
// a time, written by TMA while the next tile is computed.
constexpr int BOX_BYTES = 32 * 128;
constexpr int STAGING = EPI_WARPS * 2 * BOX_BYTES;
constexpr int SMEM = 1024 + STAGES * STAGE + STAGING + 256;
constexpr uint32_t TMEM_COLS = 512;                  // two accumulators of 256 columns
constexpr uint32_t IDESC = umma_idesc_e4m3(PT, PT);
static_assert(SMEM <= 227 * 1024 && STAGES % 2 == 0, "shared memory; stages in turn");
}  // namespace f8p

// Two boxes of R, 32 rows x (128 bytes of columns) each, from column `col`.
template <typename T>
__device__ __forceinline__ void f8_load_residual(const CUtensorMap* rmap, uint8_t* buf, uint64_t* bar,
                                                 int col, int row0) {
    constexpr int COLS = 32 * Vec<T>::N / 4;         // 128 bytes: 64 columns, or 32 of fp32
    mbar_arrive_expect_tx(bar, 2 * f8p::BOX_BYTES);
    tma_load_2d(buf, rmap, bar, col, row0);
    tma_load_2d(buf + f8p::BOX_BYTES, rmap, bar, col + COLS, row0);
}

// One warp's 32 rows x 128 columns -> Y (+ R) through `buf` (two boxes). With R, its first two
// boxes are on their way to buf already (f8_load_residual on `bar`, whose phase is r_phase).
// Boxes and rows past Y's edges are dropped by TMA. False if a wait gave up.
template <typename T>
__device__ __forceinline__ bool f8_store_boxes(const CUtensorMap* ymap, const CUtensorMap* rmap,
                                               bool res, int n_tok, int d_out, int row0, int col0,
                                               const uint64_t (&acc)[f8p::HN / 2], uint8_t* buf,
                                               uint64_t* bar, uint32_t& r_phase, int* status,
                                               volatile int* abort_flag) {
    constexpr int N = Vec<T>::N, COLS = 8 * N, ROUND = 2 * COLS;
    const int lane = lane_id();
#pragma unroll
    for (int c0 = 0; c0 < f8p::HN; c0 += ROUND) {
        if (c0 > 0) {                                // fp32: the second round reuses the boxes
            if (lane == 0) {
                bulk_wait_read<0>();
                if (res) f8_load_residual<T>(rmap, buf, bar, col0 + c0, row0);
            }
            __syncwarp();
        }
        if (res) {
            if (!f8_warp_wait(bar, r_phase, status, abort_flag)) return false;
            r_phase ^= 1;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {               // 16-byte pieces of the row
            uint8_t* at = buf + (i >> 3) * f8p::BOX_BYTES + lane * 128 + (((i & 7) ^ (lane & 7)) << 4);
            float v[N];
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = f32x2_get(acc[(c0 + i * N + e) / 2], e & 1);
            if (res) {
                float f[N];
                Vec<T>::unpack(*reinterpret_cast<const uint4*>(at), f);
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += f[e];
            }
            *reinterpret_cast<uint4*>(at) = Vec<T>::pack(v);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < n_tok) {             // whole boxes past the edge are not issued
            if (col0 + c0 < d_out) tma_store_2d(ymap, buf, col0 + c0, row0);
            if (col0 + c0 + COLS < d_out)
                tma_store_2d(ymap, buf + f8p::BOX_BYTES, col0 + c0 + COLS, row0);
            bulk_commit();
        }
    }
    return true;
}

template <typename T>
__global__ void __launch_bounds__(f8p::THREADS, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
                    const __grid_constant__ CUtensorMap ymap, const __grid_constant__ CUtensorMap rmap,
                    const F8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* staging = smem + f8p::STAGES * f8p::STAGE;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + f8p::STAGING);   // [STAGES] leader
    uint64_t* empty = full + f8p::STAGES;            // [STAGES] each CTA
    uint64_t* acc_full = empty + f8p::STAGES;        // [2] each CTA
    uint64_t* acc_empty = acc_full + 2;              // [2] leader: both CTAs have read it
    uint64_t* drained = acc_empty + 2;               // [2] leader, one per issuer
    uint64_t* r_full = drained + 2;                  // [EPI_WARPS] each CTA: a warp's part of R
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(r_full + f8p::EPI_WARPS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_id(), lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < f8p::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * f8p::EPI_WARPS);
            mbar_init(&drained[b], 1);
        }
        for (int w = 0; w < f8p::EPI_WARPS; ++w) mbar_init(&r_full[w], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&wmap);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, f8p::TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();     // both CTAs' barriers exist before either CTA signals the other's
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < f8p::EPI_WARP0) {
        regs_shrink<f8p::REGS_IO>();
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int it = 0;
            for (int t = cluster; t < p.n_tiles && !*abort_flag; t += n_clusters) {
                int m0, n0;
                f8_tile(p, t, f8p::PT, f8p::PT, m0, n0);
                m0 += f8p::BM * static_cast<int>(rank);
                n0 += f8p::BNC * static_cast<int>(rank);
                for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                    const int st = it % f8p::STAGES;
                    if (!mbar_wait(&empty[st], ((it / f8p::STAGES) & 1) ^ 1)) {
                        set_status(p.status, GPTQ_ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t* sa = smem + st * f8p::STAGE;
                    if (leader) mbar_arrive_expect_tx(&full[st], 2 * f8p::STAGE);
                    const uint32_t fb = mapa_shared(smem_u32(&full[st]), 0);
                    tma_load_2d_pair(sa, &xmap, fb, kb * f8p::BK, m0);
                    tma_load_2d_pair(sa + f8p::A_BYTES, &wmap, fb, kb * f8p::BK, n0);
                }
            }
            // the leader's stage barriers count both CTAs' bytes: once it has seen the last
            // stages complete, no copy of either CTA is still writing shared memory
            if (leader) {
                const int n_tail = it < f8p::STAGES ? it : f8p::STAGES;
                for (int k = it - n_tail; k < it; ++k) {
                    if (!mbar_wait(&full[k % f8p::STAGES], (k / f8p::STAGES) & 1)) {
                        set_status(p.status, GPTQ_ERR_TIMEOUT);
                        *abort_flag = 1;
                    }
                }
            }
        } else if ((warp == 1 || warp == 2) && leader && lane == 0) {
            // ---------------- MMA issuers (leader), every other block each ----------------
            const int b = warp - 1;
            const int per_tile = p.n_kb;
            const int mine = cluster < p.n_tiles ? (p.n_tiles - 1 - cluster) / n_clusters + 1 : 0;
            const long long blocks = static_cast<long long>(mine) * per_tile;
            bool ok = true;
            int st = b;
            uint32_t st_phase = 0, acc_phase = 1;
            for (long long it = b; it < blocks && !*abort_flag; it += 2) {
                if (!mbar_wait(&full[st], st_phase) || !mbar_wait(&acc_empty[b], acc_phase)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * f8p::PT);
                const uint32_t s0 = smem_u32(smem + st * f8p::STAGE);
#pragma unroll
                for (int kk = 0; kk < f8p::BK / 32; ++kk)
                    umma_f8_pair(d_tmem, umma_desc_sw128(s0 + kk * 32, 16, 1024),
                                 umma_desc_sw128(s0 + f8p::A_BYTES + kk * 32, 16, 1024), f8p::IDESC,
                                 kk > 0 ? 1u : 0u);
                umma_commit_pair_mc(&acc_full[b], 0x3);
                umma_commit_pair_mc(&empty[st], 0x3);
                acc_phase ^= 1;
                st += 2;
                if (st >= f8p::STAGES) {       // STAGES is even: both issuers keep their parity
                    st -= f8p::STAGES;
                    st_phase ^= 1;
                }
            }
            if (!ok) {
                set_status(p.status, GPTQ_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            // every MMA must have finished before either CTA releases TMEM or leaves
            umma_commit_pair_mc(&drained[b], 0x1);
            if (!mbar_wait(&drained[b], 0)) set_status(p.status, GPTQ_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        // ---------------- promotion (both CTAs, their own tokens) ----------------
        regs_grow<f8p::REGS_EPI>();
        const int q = warp & 3, h = (warp - f8p::EPI_WARP0) >> 2;
        const int row_in = f8p::BM * static_cast<int>(rank) + 32 * q;
        const uint32_t t_half = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                static_cast<uint32_t>(h * f8p::HN);
        const int ew = warp - f8p::EPI_WARP0;
        uint8_t* buf = staging + ew * 2 * f8p::BOX_BYTES;
        uint64_t* r_bar = &r_full[ew];
        uint32_t r_phase = 0;
        const bool boxes = p.vec_ok != 0, res = p.R != nullptr;
        int it = 0;
        bool stop = false;
        for (int t = cluster; t < p.n_tiles && !stop; t += n_clusters) {
            int m0, n0;
            f8_tile(p, t, f8p::PT, f8p::PT, m0, n0);
            const int col0 = n0 + f8p::HN * h;
            if (boxes && res && lane == 0) {
                bulk_wait_read<0>();                 // the last tile has left the boxes
                f8_load_residual<T>(&rmap, buf, r_bar, col0, m0 + row_in);
            }
            uint64_t acc[f8p::HN / 2];
#pragma unroll
            for (int k = 0; k < f8p::HN / 2; ++k) acc[k] = 0;
            const float* sx = p.sx + min(m0 + row_in + lane, p.n_tok - 1);
            const float* sw = p.sw + static_cast<int64_t>(min(col0, p.d_out - 1) / 128) * p.n_kb;
            float sx_next = __ldg(sx), sw_next = __ldg(sw);
            for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                const int b = it & 1;
                const uint32_t f = __float_as_uint(sx_next * sw_next);
                if (kb + 1 < p.n_kb) {
                    sx += p.n_tok;
                    sx_next = __ldg(sx);
                    sw_next = __ldg(sw + kb + 1);
                }
                if (!f8_warp_wait(&acc_full[b], (it >> 1) & 1, p.status, abort_flag)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint32_t t_addr = t_half + static_cast<uint32_t>(b * f8p::PT);
                // 128 columns in four loads; the accumulator is handed back as soon as the last
                // has arrived, before the last two are added
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(t_addr, r[0]);
                tmem_ld_32x32b_x32(t_addr + 32, r[1]);
                tmem_ld_wait_for(r[0]);
                tmem_ld_use(r[1]);
                f8_promote<32>(acc, r[0], f32x2(f, f));
                tmem_ld_32x32b_x32(t_addr + 64, r[0]);
                f8_promote<32>(acc + 16, r[1], f32x2(f, f));
                tmem_ld_32x32b_x32(t_addr + 96, r[1]);
                tmem_ld_wait_for(r[0]);
                tmem_ld_use(r[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive_relaxed(&acc_empty[b]);
                    else mbar_arrive_relaxed_cluster(mapa_shared(smem_u32(&acc_empty[b]), 0));
                }
                f8_promote<32>(acc + 32, r[0], f32x2(f, f));
                f8_promote<32>(acc + 48, r[1], f32x2(f, f));
            }
            if (stop) break;
            if (boxes) {
                if (!res) {
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                }
                stop = !f8_store_boxes<T>(&ymap, &rmap, res, p.n_tok, p.d_out, m0 + row_in, col0, acc,
                                          buf, r_bar, r_phase, p.status, abort_flag);
            } else {
                f8_store<T, f8p::HN>(p, m0 + row_in + lane, col0, acc);
            }
        }
        // a residual that was asked for and not used (after a timeout) must have landed
        if (boxes && res && stop && lane == 0) mbar_wait(r_bar, r_phase);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();     // neither CTA leaves while the pair's MMAs, copies or arrivals may touch it
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, f8p::TMEM_COLS);
}

template <typename T>
struct F8MapType;
template <>
struct F8MapType<__half> {
    static constexpr CUtensorMapDataType value = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
};
template <>
struct F8MapType<__nv_bfloat16> {
    static constexpr CUtensorMapDataType value = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
};
template <>
struct F8MapType<float> {
    static constexpr CUtensorMapDataType value = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
};

template <typename T>
static gptq_status fp8_pair_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                   cudaStream_t s) {
    GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_pair_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, f8p::SMEM));
    // the warpgroups' register shares add up to what a launch with REGS per thread has
    cudaFuncAttributes fa;
    GPTQ_CUDA_TRY(cudaFuncGetAttributes(&fa, fp8_pair_kernel<T>));
    if (fa.numRegs < f8p::REGS) return GPTQ_ERR_UNSUPPORTED;
    CUtensorMap xmap, wmap;
    GPTQ_TRY(encode_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(X8),
                                  p.d_in, p.n_tok, p.d_in, f8p::BK, f8p::BM,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    GPTQ_TRY(encode_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(W8),
                                  p.d_in, p.d_out, p.d_in, f8p::BK, f8p::BNC,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    CUtensorMap ymap{}, rmap{};
    if (p.vec_ok) {
        const uint64_t row = static_cast<uint64_t>(p.d_out) * sizeof(T);
        GPTQ_TRY(encode_tensor_map_2d(&ymap, F8MapType<T>::value, p.Y, p.d_out, p.n_tok, row,
                                      128 / sizeof(T), 32, CU_TENSOR_MAP_SWIZZLE_128B));
        if (p.R)
            GPTQ_TRY(encode_tensor_map_2d(&rmap, F8MapType<T>::value, const_cast<void*>(p.R), p.d_out,
                                          p.n_tok, row, 128 / sizeof(T), 32,
                                          CU_TENSOR_MAP_SWIZZLE_128B));
    }
    p.n_mt = (p.n_tok - 1) / f8p::PT + 1;
    p.n_nt = (p.d_out - 1) / f8p::PT + 1;
    GPTQ_TRY(f8_tiles(p));
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    cfg.blockDim = dim3(f8p::THREADS);
    cfg.dynamicSmemBytes = f8p::SMEM;
    cfg.stream = s;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(p.n_tiles, num_sms() / 2)));
    GPTQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, fp8_pair_kernel<T>, xmap, wmap, ymap, rmap, p));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

template <typename T>
static gptq_status fp8_linear_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                     cudaStream_t s) {
    p.vec_ok = p.d_out % Vec<T>::N == 0;
    const long long pair_tiles = static_cast<long long>((p.n_tok - 1) / f8p::PT + 1) *
                                 ((p.d_out - 1) / f8p::PT + 1);
    if (p.n_tok > 128 && 2 * pair_tiles >= num_sms()) return fp8_pair_launch<T>(X8, W8, p, s);
    return fp8_gemm_launch<T>(X8, W8, p, s);
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
        case GPTQ_DTYPE_F16: return gq::fp8_linear_launch<__half>(X8, W8, p, s);
        case GPTQ_DTYPE_BF16: return gq::fp8_linear_launch<__nv_bfloat16>(X8, W8, p, s);
        default: return gq::fp8_linear_launch<float>(X8, W8, p, s);
    }
}
