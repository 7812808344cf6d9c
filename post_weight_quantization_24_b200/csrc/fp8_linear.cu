// Y = Xhat * What^T (+ R) from e4m3 codes with one scale per token and 128 channels (X) and per
// 128 x 128 block (W), on the 5th-generation tensor cores:
//   Y[t][o] = sum_b sx[b][t] * sw[o/128][b] * (sum_{c in block b} X8[t][c] * W8[o][c]) + R[t][o].
//
// The scales change every 128 channels, so the tensor cores sum one block at a time from zero
// (4 x tcgen05.mma kind::f8f6f4 of K = 32, fp32 accumulator in TMEM) and the sum over blocks
// is kept in registers: acc = fma(partial, sx*sw, acc), rounded to nearest.
//
// Two kernels, both fed by TMA (128-byte swizzle) with bounded waits everywhere: on timeout a
// kernel records GPTQ_ERR_TIMEOUT, drains its copies and MMAs, frees TMEM and returns. Tokens and
// channels past the edges are zero-filled by TMA and not stored.
//   fp8_pair_kernel    256 tokens x 256 channels per CTA pair, for calls with enough such tiles to
//                      fill the GPU. 16384 tokens, 11008 -> 4096, fp16 with residual: 0.82 to 0.86
//                      ms back to back (1.7 to 1.8 PFLOP/s), 0.77 ms in short runs. The
//                      promotion's multiply-adds bound it: 1035 cycles per block at 1.52 GHz
//                      with them; without them 690 to 740 at 1.30 to 1.41 GHz (0.63 ms, at the
//                      power limit), as with TMA and MMAs alone.
//   fp8_stream_kernel  128 channels x 16 to 128 tokens per CTA, the input channels split over a
//                      cluster: for all other calls. 1 token, 4096 -> 4096: 7.2 us; 37 tokens,
//                      11008 -> 4096, bf16 with residual: 15.7 us, about 4 us of them fixed
//                      (set-up, first loads, the join) and the rest at 4 to 5 TB/s of weights.
#include <algorithm>
#include <atomic>

#include "internal.cuh"
#include "vec.cuh"

namespace gq {

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
    long long wait_limit; // cycles after which a wait gives up
    int stall_rank;       // test switch: the CTA of a cluster whose producer gives up, or -1
};

// Test switch for the give-up paths (set by gptq_test_stall_fp8, read when a call is enqueued): the
// producer of one CTA in each cluster behaves as if its wait for a stage had run out, a few
// blocks into its work. Copies, MMAs and sums are in flight then, in its CTA and in the others,
// whose own waits give up after STALL_LIMIT_CYCLES.
static std::atomic<int> g_fp8_stall{-1};
constexpr long long STALL_LIMIT_CYCLES = 2000000;   // about 1 ms

gptq_status fp8_stall_set(int rank) {
    g_fp8_stall.store(rank < 0 ? -1 : rank);
    return GPTQ_OK;
}

// Test switch: calls behave as on a build whose pair kernel cannot be launched.
static std::atomic<int> g_fp8_no_pair{0};

gptq_status fp8_no_pair_set(int on) {
    g_fp8_no_pair.store(on ? 1 : 0);
    return GPTQ_OK;
}

// NC accumulated columns of one row -> Y (+ R), value by value: for rows that do not all start on
// 16-byte boundaries. A warp's lanes are 32 rows, so each access touches 32 sectors for 64 or 128
// useful bytes: 4096 tokens, 2048 -> 4095, fp16, take 201 us (242 with R) against 47 (53) for 2048 ->
// 4096.
template <typename T, int NC>
__device__ __forceinline__ void f8_store(const F8Params& p, int row, int col0,
                                         const uint64_t (&acc)[NC / 2]) {
    if (row >= p.n_tok) return;
    const int64_t off = static_cast<int64_t>(row) * p.d_out + col0;
    T* y = static_cast<T*>(p.Y) + off;
    const T* r = p.R ? static_cast<const T*>(p.R) + off : nullptr;
    const int left = p.d_out - col0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (c < left)
            y[c] = Vec<T>::from_float(f32x2_get(acc[c / 2], c & 1) +
                                      (r ? Vec<T>::to_float(r[c]) : 0.0f));
    }
}

// acc += f * (NC/2 pairs of partial sums)
template <int NC>
__device__ __forceinline__ void f8_promote(uint64_t* acc, const uint32_t (&r)[NC], uint64_t f) {
#pragma unroll
    for (int k = 0; k < NC / 2; ++k) fma_f32x2(acc[k], f32x2(r[2 * k], r[2 * k + 1]), f);
}

// Wait of a whole warp, every lane on the barrier itself: true if it completed for all of them, else
// the timeout is recorded. The lanes leave together with one answer, because what follows needs them
// all. With WATCH the wait also ends once another wait of the CTA has given up, which a caller that
// carries on after a give-up needs; to test the flag ahead of the wait instead would let each lane
// decide by itself, and could send some past a vote that the others are in.
template <bool WATCH = false>
__device__ __forceinline__ bool f8_warp_wait(uint64_t* bar, uint32_t parity, const F8Params& p,
                                             volatile int* abort_flag) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const long long t0 = clock64();
        while (!(ok = mbar_try_wait(bar, parity)) && clock64() - t0 <= p.wait_limit) {
            if (WATCH && *abort_flag) break;
        }
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    set_status(p.status, GPTQ_ERR_TIMEOUT);
    *abort_flag = 1;
    return false;
}

// ---------------------------------------------------------------------------------------
// Streaming kernel: Y^T tiles of 128 channels x NT tokens, the weights as the MMA's M operand, so
// that a few tokens cost a narrow N instead of an M of 128 rows. A cluster of S CTAs splits the
// tile's input channels. Each CTA streams its part of the weights (16 KB per block) through a ring of
// stages and sends its partial sums to the CTAs that own their tokens (st.async into their shared
// memory, counted on an mbarrier there), which add them in rank order, so equal inputs give equal
// bits. Nobody reads another CTA's memory, so no cluster barrier (1100 cycles each) is left but
// one whose latency the main loop covers: 16 tokens, 11008 -> 4096, took 11.7 us against 12.9 with
// sums read between two barriers (11.4 now). Two CTAs fit an SM, one for 128 tokens (128 tokens, 11008
// -> 4096, 17.5 us now, took 24 us with one of 6 stages, 31 us with two of 3, in an earlier form).
// With tokens as M and no split the 37-token call above took 43.6 us.
//   warp 0    TMA producer            warps 1, 2  MMA issuers, every other block each
//   warps 3-  promotion: a thread owns one channel and EC tokens. The factors sx*sw (one per token
//             and block) are put into shared memory for FBLK blocks at a time, which exposes
//             their latency once instead of once per block.
// ---------------------------------------------------------------------------------------
namespace f8s {
constexpr int BM = 128, BK = 128;
template <int NT>
struct Cfg {
    static constexpr int PER_SM = NT == 128 ? 1 : 2;              // CTAs that fit an SM
    static constexpr int STAGES = NT == 16 ? 5 : NT == 32 ? 4 : NT == 64 ? 3 : 4;
    static constexpr int A_BYTES = BM * BK, STAGE = A_BYTES + NT * BK;
    static constexpr int ACCS = NT >= 64 ? 2 : 4;
    static constexpr uint32_t TMEM_COLS = ACCS * NT;
    static constexpr int EC = NT <= 32 ? 16 : 32, EPI_WARPS = 4 * (NT / EC);
    static constexpr int EPI_THREADS = EPI_WARPS * 32, THREADS = 96 + EPI_THREADS;
    static constexpr int FBLK = NT >= 64 ? 16 : 32;              // blocks of factors kept
    static constexpr int RECV = NT * BM * 4;                     // the cluster's sums of this CTA's tokens
    static constexpr int SMEM = 1024 + STAGES * STAGE + RECV + FBLK * NT * 4 + 256;
    static constexpr int BARRIERS = 2 * STAGES + 2 * ACCS + 3;   // full, empty, acc_full, acc_empty, ...
    static constexpr uint32_t IDESC = umma_idesc_e4m3(BM, NT);
    static_assert(FBLK * NT == 4 * EPI_THREADS, "four factors per promotion thread");
    static_assert(BARRIERS <= 32, "a lane sets up each");
    static_assert(PER_SM * (SMEM + 1024) <= 228 * 1024, "CTAs per SM");
    // An issuer waits for its accumulator first: that block it - ACCS has been added tells that the
    // stage's last load (block it - STAGES) landed, so a parity wait on the stage cannot take the
    // phase before last for the last. An accumulator belongs to one issuer for the same reason.
    static_assert(ACCS % 2 == 0 && STAGES >= ACCS, "phases in order");
};
}  // namespace f8s

template <typename T, int NT>
__global__ void __launch_bounds__(f8s::Cfg<NT>::THREADS, f8s::Cfg<NT>::PER_SM)
    fp8_stream_kernel(const __grid_constant__ CUtensorMap xmap,
                      const __grid_constant__ CUtensorMap wmap, const F8Params p, int splits) {
    using C = f8s::Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* recv = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);         // [rank][token][channel]
    float* factors = recv + C::RECV / 4;                                         // [FBLK][NT]
    uint64_t* full = reinterpret_cast<uint64_t*>(factors + C::FBLK * NT);
    uint64_t* empty = full + C::STAGES;
    uint64_t* acc_full = empty + C::STAGES;
    uint64_t* acc_empty = acc_full + C::ACCS;
    uint64_t* drained = acc_empty + C::ACCS;
    uint64_t* recv_full = drained + 2;     // the last of BARRIERS in a row
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(recv_full + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = warp_id(), lane = lane_id();
    const int rank = static_cast<int>(cluster_ctarank());
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int t0 = (tile % p.n_mt) * NT, c0 = (tile / p.n_mt) * f8s::BM;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.n_kb) * rank / splits);
    const int n_kb = static_cast<int>(static_cast<int64_t>(p.n_kb) * (rank + 1) / splits) - kb0;
    auto load = [&](int it) {      // block it of this CTA into its stage
        const int st = it % C::STAGES;
        uint8_t* sa = smem + st * C::STAGE;
        const int x = (kb0 + it) * f8s::BK;
        mbar_arrive_expect_tx(&full[st], C::STAGE);
        tma_load_2d(sa, &wmap, &full[st], x, c0);
        tma_load_2d(sa + C::A_BYTES, &xmap, &full[st], x, t0);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_cycles(bar, parity, p.wait_limit);
    };
    const int first = min(C::STAGES, n_kb);
    // The promotion threads' scales of blocks it0 .. it0 + FBLK - 1, four values each, all asked for at
    // once (entries past the last block or token repeat the last: they are not used).
    const int e = static_cast<int>(threadIdx.x) - 96;  // promotion thread
    float fx[4], fw[4];
    auto fetch_factors = [&](int it0) {
        const float* sx = p.sx + static_cast<int64_t>(kb0) * p.n_tok + t0;
        const float* sw = p.sw + static_cast<int64_t>(c0 / 128) * p.n_kb + kb0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = e + u * C::EPI_THREADS;
            const int kb = min(it0 + i / NT, n_kb - 1), t = min(i % NT, p.n_tok - 1 - t0);
            fx[u] = __ldg(sx + static_cast<int64_t>(kb) * p.n_tok + t);
            fw[u] = __ldg(sw + kb);
        }
    };
    // the first loads leave while the rest is still being set up
    if (warp == 0) {
        if (lane < C::BARRIERS) {
            const int a = lane - 2 * C::STAGES - C::ACCS;            // acc_empty's number, if it is one
            mbar_init(&full[lane], a >= 0 && a < C::ACCS ? C::EPI_WARPS : 1);
            fence_mbar_init();
        }
        __syncwarp();
        if (lane == 0) {
            *abort_flag = 0;
            mbar_arrive_expect_tx(recv_full, C::RECV);
            pdl_wait();
            for (int it = 0; it < first; ++it) load(it);
        }
    } else if (warp >= 3) {
        pdl_wait();
        fetch_factors(0);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_arrive();   // this CTA's barriers exist; waited for before anything is sent
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int it = first;
            for (; it < n_kb && !*abort_flag; ++it) {
                if ((it == C::STAGES + 1 && rank == p.stall_rank) ||
                    !wait(&empty[it % C::STAGES], ((it / C::STAGES) & 1) ^ 1)) {
                    set_status(p.status, GPTQ_ERR_TIMEOUT);
                    *abort_flag = 1;
                    break;
                }
                load(it);
            }
            const int n_tail = it < C::STAGES ? it : C::STAGES;
            for (int k = it - n_tail; k < it; ++k) {
                if (!wait(&full[k % C::STAGES], (k / C::STAGES) & 1)) {
                    set_status(p.status, GPTQ_ERR_TIMEOUT);
                    *abort_flag = 1;
                }
            }
        }
        __syncwarp();
    } else if (warp < 3) {
        if (lane == 0) {
            bool ok = true;
            for (int it = warp - 1; it < n_kb && !*abort_flag; it += 2) {
                const int st = it % C::STAGES, b = it % C::ACCS;
                if (!wait(&acc_empty[b], ((it / C::ACCS) & 1) ^ 1) ||
                    !wait(&full[st], (it / C::STAGES) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(b * NT);
                const uint32_t s0 = smem_u32(smem + st * C::STAGE);
#pragma unroll
                for (int kk = 0; kk < f8s::BK / 32; ++kk) {
                    // K-major rows of 128 B; a k-step of 32 codes is 32 B along the row
                    umma_f8(d_tmem, umma_desc_sw128(s0 + kk * 32, 16, 1024),
                            umma_desc_sw128(s0 + C::A_BYTES + kk * 32, 16, 1024), C::IDESC,
                            kk > 0 ? 1u : 0u);
                }
                umma_commit(&acc_full[b]);
                umma_commit(&empty[st]);
            }
            if (!ok) {
                set_status(p.status, GPTQ_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            umma_commit(&drained[warp - 1]);
            if (!wait(&drained[warp - 1], 0)) set_status(p.status, GPTQ_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, g = (warp - 3) >> 2;       // channel quarter, token group
        const uint32_t t_addr0 = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                 static_cast<uint32_t>(g * C::EC);
        float acc[C::EC];
#pragma unroll
        for (int k = 0; k < C::EC; ++k) acc[k] = 0.0f;
        for (int it = 0; it < n_kb; ++it) {
            const int b = it % C::ACCS;
            if (it % C::FBLK == 0) {
                // the next FBLK blocks' factors, after everybody has used the last ones
                if (it > 0) {
                    fetch_factors(it);
                    asm volatile("bar.sync 1, %0;" ::"n"(C::EPI_THREADS) : "memory");
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) factors[e + u * C::EPI_THREADS] = fx[u] * fw[u];
                asm volatile("bar.sync 1, %0;" ::"n"(C::EPI_THREADS) : "memory");
            }
            // after a wait that gave up the loop runs out: the barriers above need every
            // promotion thread
            f8_warp_wait<true>(&acc_full[b], (it / C::ACCS) & 1, p, abort_flag);
            tc_fence_after();
            const uint32_t t_addr = t_addr0 + static_cast<uint32_t>(b * NT);
            const float* f = factors + (it % C::FBLK) * NT + g * C::EC;
#pragma unroll
            for (int j = 0; j < C::EC / 16; ++j) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(t_addr + 16 * j, r);
                tmem_ld_wait_for(r);
                if (j == C::EC / 16 - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed(&acc_empty[b]);
                }
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 f4 = *reinterpret_cast<const float4*>(f + 16 * j + k);
                    acc[16 * j + k] = fmaf(__uint_as_float(r[k]), f4.x, acc[16 * j + k]);
                    acc[16 * j + k + 1] = fmaf(__uint_as_float(r[k + 1]), f4.y, acc[16 * j + k + 1]);
                    acc[16 * j + k + 2] = fmaf(__uint_as_float(r[k + 2]), f4.z, acc[16 * j + k + 2]);
                    acc[16 * j + k + 3] = fmaf(__uint_as_float(r[k + 3]), f4.w, acc[16 * j + k + 3]);
                }
            }
        }
        // every token's sums to the CTA that owns it, as [rank][token of the owner][channel]
        const int share = NT / splits, shift = 31 - __clz(share);
        const uint32_t my_part = smem_u32(recv) +
                                 static_cast<uint32_t>((rank * share * f8s::BM + 32 * q + lane) * 4);
        __syncwarp();
        cluster_wait();
#pragma unroll
        for (int k = 0; k < C::EC; ++k) {
            const int t = g * C::EC + k, owner = t >> shift;
            st_async_b32(mapa_shared(my_part + static_cast<uint32_t>((t & (share - 1)) * f8s::BM * 4),
                                     static_cast<uint32_t>(owner)),
                         __float_as_uint(acc[k]),
                         mapa_shared(smem_u32(recv_full), static_cast<uint32_t>(owner)));
        }
        // this CTA's share of the tokens: a warp takes a token, a lane four channels
        const bool got = f8_warp_wait(recv_full, 0, p, abort_flag);
        const int col = c0 + 4 * lane;
        for (int i = warp - 3; i < share; i += C::EPI_WARPS) {
            const int row = t0 + rank * share + i;
            if (!got || row >= p.n_tok || col >= p.d_out) continue;
            const float4* x = reinterpret_cast<const float4*>(recv + i * f8s::BM) + lane;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int r = 0; r < splits; ++r) {
                const float4 y4 = x[r * share * (f8s::BM / 4)];
                v[0] += y4.x;
                v[1] += y4.y;
                v[2] += y4.z;
                v[3] += y4.w;
            }
            const int64_t off = static_cast<int64_t>(row) * p.d_out + col;
            const T* R = p.R ? static_cast<const T*>(p.R) + off : nullptr;
            T* y = static_cast<T*>(p.Y) + off;
            if (p.vec_ok) {
                struct alignas(4 * sizeof(T)) Four { T v[4]; };
                Four o;
                if (R) {
                    const Four x = *reinterpret_cast<const Four*>(R);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] += Vec<T>::to_float(x.v[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o.v[j] = Vec<T>::from_float(v[j]);
                *reinterpret_cast<Four*>(y) = o;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (col + j < p.d_out)
                        y[j] = Vec<T>::from_float(v[j] + (R ? Vec<T>::to_float(R[j]) : 0.0f));
            }
        }
    }
    if (warp < 3) {
        __syncwarp();
        cluster_wait();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
    if (*abort_flag) {
        // Sums for this CTA may still be under way: every CTA sends its own, whatever else it gave
        // up. This CTA stays until the others have sent theirs (they have left, needing nothing of
        // it, or wait here too) and until all have arrived.
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (threadIdx.x == 0) wait(recv_full, 0);
    }
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
constexpr int BAND = 8;                              // token tiles of a band
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
                                               uint64_t* bar, uint32_t& r_phase, const F8Params& p,
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
            if (!f8_warp_wait(bar, r_phase, p, abort_flag)) return false;
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

// Tiles run in bands of 8 token tiles with the token tile varying fastest, so the CTAs that run
// together share weight tiles and activation rows in L2.
__device__ __forceinline__ void f8_tile(const F8Params& p, int t, int& m0, int& n0) {
    const int per_band = f8p::BAND * p.n_nt;
    const int band = t / per_band;
    const int rem = t - band * per_band;
    const int band_m = min(f8p::BAND, p.n_mt - band * f8p::BAND);
    m0 = (band * f8p::BAND + rem % band_m) * f8p::PT;
    n0 = (rem / band_m) * f8p::PT;
}

// Block kb of a tile into stage st: this CTA's tokens and its half of the channels. Both CTAs' bytes
// complete on the leader's barrier, which the leader arms for both.
__device__ __forceinline__ void f8_pair_load(const CUtensorMap* xmap, const CUtensorMap* wmap,
                                             uint8_t* smem, uint64_t* full, bool leader, int st, int kb,
                                             int m0, int n0) {
    uint8_t* sa = smem + st * f8p::STAGE;
    if (leader) mbar_arrive_expect_tx(&full[st], 2 * f8p::STAGE);
    const uint32_t fb = mapa_shared(smem_u32(&full[st]), 0);
    tma_load_2d_pair(sa, xmap, fb, kb * f8p::BK, m0);
    tma_load_2d_pair(sa + f8p::A_BYTES, wmap, fb, kb * f8p::BK, n0);
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
    // whether this CTA and the other one have given up, and then the blocks that each has loaded
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);   // [2]
    volatile uint32_t* loaded = tmem_slot + 4;                                   // [2], by rank

    const int warp = warp_id(), lane = lane_id();
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return mbar_wait_cycles(bar, parity, p.wait_limit);
    };
    auto tell_other = [&](volatile void* at, uint32_t v) {
        st_shared_cluster_b32(mapa_shared(smem_u32(const_cast<const void*>(at)), rank ^ 1), v);
    };
    // this CTA's first token and first channel to load of tile t
    auto tile_of = [&](int t, int& m0, int& n0) {
        f8_tile(p, t, m0, n0);
        m0 += f8p::BM * static_cast<int>(rank);
        n0 += f8p::BNC * static_cast<int>(rank);
    };
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
        abort_flag[0] = abort_flag[1] = 0;
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
    pdl_wait();

    if (warp < f8p::EPI_WARP0) {
        regs_shrink<f8p::REGS_IO>();
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            int it = 0;
            for (int t = cluster; t < p.n_tiles && !*abort_flag; t += n_clusters) {
                int m0, n0;
                tile_of(t, m0, n0);
                for (int kb = 0; kb < p.n_kb; ++kb, ++it) {
                    const int st = it % f8p::STAGES;
                    if ((it == f8p::STAGES + 1 && static_cast<int>(rank) == p.stall_rank) ||
                        !wait(&empty[st], ((it / f8p::STAGES) & 1) ^ 1)) {
                        set_status(p.status, GPTQ_ERR_TIMEOUT);
                        *abort_flag = 1;
                        break;
                    }
                    f8_pair_load(&xmap, &wmap, smem, full, leader, st, kb, m0, n0);
                }
            }
            // The last stages' releases: every block that was loaded has then been multiplied, so no
            // copy is in flight, and no release is still on its way to this CTA's barriers. After a
            // give-up the copies are seen to below.
            const int n_tail = it < f8p::STAGES ? it : f8p::STAGES;
            for (int k = it - n_tail; k < it && !*abort_flag; ++k) {
                if (!wait(&empty[k % f8p::STAGES], (k / f8p::STAGES) & 1)) {
                    set_status(p.status, GPTQ_ERR_TIMEOUT);
                    *abort_flag = 1;
                }
            }
            loaded[rank] = static_cast<uint32_t>(it);
            if (*abort_flag) tell_other(abort_flag + 1, 1);
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
                if (!wait(&full[st], st_phase) || !wait(&acc_empty[b], acc_phase)) {
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
            if (!wait(&drained[b], 0)) {
                set_status(p.status, GPTQ_ERR_TIMEOUT);
                *abort_flag = 1;
            }
            if (*abort_flag) tell_other(abort_flag + 1, 1);
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
            f8_tile(p, t, m0, n0);
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
                if (!f8_warp_wait(&acc_full[b], (it >> 1) & 1, p, abort_flag)) {
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
                                          buf, r_bar, r_phase, p, abort_flag);
            } else {
                f8_store<T, f8p::HN>(p, m0 + row_in + lane, col0, acc);
            }
        }
        // a residual that was asked for and not used (after a timeout) must have landed
        if (boxes && res && stop && lane == 0) wait(r_bar, r_phase);
        if (stop && lane == 0) tell_other(abort_flag + 1, 1);
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();     // neither CTA leaves while the pair's MMAs, copies or arrivals may touch it
    tc_fence_after();
    if (const int2 gave_up = *reinterpret_cast<const int2*>(const_cast<const int*>(abort_flag));
        gave_up.x || gave_up.y) {
        // One of the two gave up, and its producer may have stopped before the other's. The one that
        // is behind (by STAGES blocks at most: a stage is released to both) loads what the other has
        // loaded, so that the leader's barriers complete for both CTAs' copies. No MMA is left to
        // read the stages.
        if (threadIdx.x == 0) tell_other(&loaded[rank], loaded[rank]);
        __syncwarp();
        cluster_sync();
        if (threadIdx.x == 0) {
            const int blocks = static_cast<int>(max(loaded[0], loaded[1]));
            for (int it = static_cast<int>(loaded[rank]); it < blocks; ++it) {
                int m0, n0;
                tile_of(cluster + it / p.n_kb * n_clusters, m0, n0);
                f8_pair_load(&xmap, &wmap, smem, full, leader, it % f8p::STAGES, it % p.n_kb, m0, n0);
            }
            if (leader)
                for (int it = max(0, blocks - f8p::STAGES); it < blocks; ++it)
                    wait(&full[it % f8p::STAGES], (it / f8p::STAGES) & 1);
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1) tmem_dealloc_pair(tmem_base, f8p::TMEM_COLS);
}

// `setup` once per device (kernel attributes belong to a device's context).
template <typename F>
static gptq_status f8_once(std::atomic<unsigned long long>& done, F&& setup) {
    int dev = 0;
    GPTQ_CUDA_TRY(cudaGetDevice(&dev));
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return GPTQ_OK;
    GPTQ_TRY(setup());
    done.fetch_or(bit, std::memory_order_release);
    return GPTQ_OK;
}

// Launch with clusters of `cluster` CTAs along x, set-up overlapped with the previous kernel's end
// (the kernels pdl_wait() before they read anything).
template <typename... KArgs, typename... Args>
static gptq_status f8_launch(void (*kernel)(KArgs...), int grid, int cluster, int threads, int smem,
                             cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    GPTQ_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, args...));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

// Ways to split the input channels of `tiles` streaming tiles, a power of two up to 8: until there is
// a CTA for every SM, as long as each keeps 2 blocks (1 token, 1024 -> 1024: 3.8 us in quarters,
// 4.6 us in halves). Where two CTAs share an SM, one more doubling pays if each keeps 8 blocks (37
// tokens, 11008 -> 4096: 15.7 us in eighths, 17.0 us in quarters), and costs with fewer (64 tokens,
// 4096 -> 4096: 10.7 us in eighths, 9.9 us in quarters).
static int f8_splits(long long tiles, int n_kb, int per_sm) {
    int splits = 1;
    while (splits < 8 &&
           ((2 * tiles * splits <= num_sms() && 4 * splits <= n_kb) ||
            (per_sm == 2 && tiles * splits < num_sms() && 16 * splits <= n_kb)))
        splits *= 2;
    return splits;
}

template <typename T, int NT>
static gptq_status fp8_stream_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                     cudaStream_t s) {
    using C = f8s::Cfg<NT>;
    static std::atomic<unsigned long long> done{0};
    GPTQ_TRY(f8_once(done, []() -> gptq_status {
        GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_stream_kernel<T, NT>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
        return GPTQ_OK;
    }));
    CUtensorMap xmap, wmap;
    GPTQ_TRY(encode_tensor_map_2d(&xmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(X8),
                                  p.d_in, p.n_tok, p.d_in, f8s::BK, NT, CU_TENSOR_MAP_SWIZZLE_128B));
    GPTQ_TRY(encode_tensor_map_2d(&wmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, const_cast<uint8_t*>(W8),
                                  p.d_in, p.d_out, p.d_in, f8s::BK, f8s::BM,
                                  CU_TENSOR_MAP_SWIZZLE_128B));
    p.n_mt = (p.n_tok - 1) / NT + 1;
    p.n_nt = (p.d_out - 1) / f8s::BM + 1;
    const long long tiles = static_cast<long long>(p.n_mt) * p.n_nt;
    const int splits = f8_splits(tiles, p.n_kb, C::PER_SM);
    if (tiles * splits > 0x7FFFFFFF) return GPTQ_ERR_ARG;
    return f8_launch(fp8_stream_kernel<T, NT>, static_cast<int>(tiles) * splits, splits, C::THREADS,
                     C::SMEM, s, xmap, wmap, p, splits);
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

// Whether this device can run the pair kernel: the warpgroups' register shares add up to what a
// launch with REGS per thread has, which is the compiler's to give. Without it the streaming kernel
// serves every call.
template <typename T>
static gptq_status fp8_pair_usable(bool* usable) {
    static std::atomic<unsigned long long> done{0}, too_few{0};
    int dev = 0;
    GPTQ_CUDA_TRY(cudaGetDevice(&dev));
    const unsigned long long bit = 1ull << (dev & 63);
    GPTQ_TRY(f8_once(done, [&]() -> gptq_status {
        GPTQ_CUDA_TRY(cudaFuncSetAttribute(fp8_pair_kernel<T>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, f8p::SMEM));
        cudaFuncAttributes fa;
        GPTQ_CUDA_TRY(cudaFuncGetAttributes(&fa, fp8_pair_kernel<T>));
        if (fa.numRegs < f8p::REGS) too_few.fetch_or(bit);
        return GPTQ_OK;
    }));
    *usable = !(too_few.load() & bit) && !g_fp8_no_pair.load();
    return GPTQ_OK;
}

template <typename T>
static gptq_status fp8_pair_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                   cudaStream_t s) {
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
    // tile numbers (with a launch's stride added) stay within 31 bits
    const long long tiles = static_cast<long long>(p.n_mt) * p.n_nt;
    if (tiles > 0x7FFF0000 || f8p::BAND * static_cast<long long>(p.n_nt) > 0x7FFF0000)
        return GPTQ_ERR_ARG;
    p.n_tiles = static_cast<int>(tiles);
    return f8_launch(fp8_pair_kernel<T>, 2 * std::min(p.n_tiles, num_sms() / 2), 2, f8p::THREADS,
                     f8p::SMEM, s, xmap, wmap, ymap, rmap, p);
}

template <typename T>
static gptq_status fp8_linear_launch(const uint8_t* X8, const uint8_t* W8, F8Params& p,
                                     cudaStream_t s) {
    p.vec_ok = p.d_out % Vec<T>::N == 0;
    const long long pair_tiles = static_cast<long long>((p.n_tok - 1) / f8p::PT + 1) *
                                 ((p.d_out - 1) / f8p::PT + 1);
    if (p.n_tok > 64) {
        // Blocks of 128 input channels one after the other, a wave of pair tiles a little faster than
        // one of 128 x 128 streaming tiles (0.55 and 0.53 to 0.6 us per block over 86 blocks, 0.68 us
        // each over 32, start and end of the call included), so the streaming kernel is taken where
        // splitting d_in or a partial wave saves more than the 5 to 6 of the rule. 256 tokens: 11008
        // -> 4096 26 us, with pairs 49 us; 4096 -> 11008 42 us, with pairs 22 us. 384 tokens, 11008
        // -> 4096: 45 us, with pairs, which the rule takes, 48 us.
        const long long pair_waves = (pair_tiles + num_sms() / 2 - 1) / (num_sms() / 2);
        const long long tiles = static_cast<long long>((p.n_tok - 1) / 128 + 1) * ((p.d_out - 1) / 128 + 1);
        const int splits = f8_splits(tiles, p.n_kb, 1);
        const long long waves = (tiles * splits + num_sms() - 1) / num_sms();
        if (5 * pair_waves * p.n_kb <= 6 * waves * ((p.n_kb + splits - 1) / splits)) {
            bool usable = false;
            GPTQ_TRY(fp8_pair_usable<T>(&usable));
            if (usable) return fp8_pair_launch<T>(X8, W8, p, s);
        }
    }
    if (p.n_tok <= 16) return fp8_stream_launch<T, 16>(X8, W8, p, s);
    if (p.n_tok <= 32) return fp8_stream_launch<T, 32>(X8, W8, p, s);
    if (p.n_tok <= 64) return fp8_stream_launch<T, 64>(X8, W8, p, s);
    return fp8_stream_launch<T, 128>(X8, W8, p, s);
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
    // Y is written while other tiles are still read: R may be Y itself (every value is read by
    // whoever writes it), and nothing else may share memory with Y
    const int64_t n_kb = (d_in + 127) / 128;
    const int64_t y_bytes = gq::range_bytes(n_tokens * d_out, y_dtype == GPTQ_DTYPE_F32 ? 4 : 2);
    if ((R != Y && gq::overlap(Y, y_bytes, R, y_bytes)) ||
        gq::overlap(Y, y_bytes, X8, n_tokens * d_in) ||
        gq::overlap(Y, y_bytes, W8, static_cast<int64_t>(d_out) * d_in) ||
        gq::overlap(Y, y_bytes, x_scales, 4 * n_kb * n_tokens) ||
        gq::overlap(Y, y_bytes, w_scales, 4 * n_kb * ((static_cast<int64_t>(d_out) + 127) / 128)))
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
    p.stall_rank = gq::g_fp8_stall.load();
    p.wait_limit = p.stall_rank < 0 ? gq::kWaitLimitCycles : gq::STALL_LIMIT_CYCLES;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (y_dtype) {
        case GPTQ_DTYPE_F16: return gq::fp8_linear_launch<__half>(X8, W8, p, s);
        case GPTQ_DTYPE_BF16: return gq::fp8_linear_launch<__nv_bfloat16>(X8, W8, p, s);
        default: return gq::fp8_linear_launch<float>(X8, W8, p, s);
    }
}
