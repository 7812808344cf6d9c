// The quantised key/value cache: keys and values get the group min-max quantizer of quant.cuh
// (per token and head, groups along head_dim) as they are written into a paged cache, and are
// read back as scale * (code - zero).
//
// Both kernels move each byte once. 16384 tokens x 32 heads x 128, 4 bits, bf16: writing takes 60 us
// (5.7 TB/s, 0.87 of the copy rate), reading 59 us (5.8 TB/s); 131072 tokens x 8 heads x 128 read in
// 113 us (6.1 TB/s, 78 % of the bytes are writes). Writing from fp32, 8 bits: 107 us (6.3 TB/s). Groups
// of 16 write in 85 us (four sets of fp64 scalars per lane); rows that are no multiple of 256 elements
// go pass by pass (16384 x 3 x 80: 13 us, 1.6 TB/s, read in 8). A decode step's few tokens are bound
// by launch latency (3 us on the device).
//
// A token's heads lie together in the cache, so its n_heads * head_dim elements are one contiguous
// row in every array: `wc` chunks of 8 elements, of which a warp takes 32 consecutive ones per
// pass. Where rows are whole multiples of 128, 64 or 32 chunks (1024, 512 or 256 elements), it
// takes four, two or one passes of a token's keys and the same of its values at a time (U = 8, 4
// or 2 passes), which shares the token's addresses among them and the work on the groups' scalars,
// and keeps 16 U bytes per lane in flight. Other widths go pass by pass over the ends of plane
// rows (token 0's keys, token 0's values, token 1's keys, ...; U = 1). A group is 2 to 32
// consecutive chunks and never straddles a pass, because it divides both.
#include <algorithm>
#include <type_traits>

#include "internal.cuh"
#include "quant.cuh"
#include "vec.cuh"

namespace gq {

struct KvParams {
    int64_t n_slots;       // slots of one plane (keys; the values' plane follows)
    int width, wc;         // elements and 8-element chunks of a token's row
    int ng;                // groups of a row
    int tpg_shift;         // log2 of the chunks per group (1 .. 5)
    uint8_t* codes;
    uint16_t* scales;
    uint16_t* zeros;
    int* status;
};

constexpr int kKvThreads = 128;

// fp32 goes out as one store of 32 bytes per lane where rows start on such boundaries: two of 16,
// each touching half of every 32-byte sector, took 15 % more.
__device__ __forceinline__ void kv_store8(float* p, const float* v, int wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                     "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = Vec<float>::pack(v);
        *(reinterpret_cast<uint4*>(p) + 1) = Vec<float>::pack(v + 4);
    }
}
template <typename T>
__device__ __forceinline__ void kv_store8(T* p, const float* v, int) {
    *reinterpret_cast<uint4*>(p) = Vec<T>::pack(v);
}

constexpr uint16_t kHalfNan = 0x7E00;
constexpr float kMagicInt = 12582912.0f;   // 1.5 * 2^23: adding it rounds to an integer, half to even

// A group's grid as the code loop uses it: 1/scale, and what turns the bits of a rounded quotient
// into its code (scale and zero for the exact decision only).
struct KvGrid {
    float inv;
    int to_code;
    float scale, zero;
};

// Eight codes (0 .. MAXQ) packed. BITS == 4: one word; 8: two.
template <int BITS>
__device__ __forceinline__ uint2 pack_codes(const int* q) {
    if (BITS == 4)
        return make_uint2(((q[0] + (q[1] << 4)) + ((q[2] + (q[3] << 4)) << 8)) +
                              (((q[4] + (q[5] << 4)) + ((q[6] + (q[7] << 4)) << 8)) << 16),
                          0);
    return make_uint2((q[0] + (q[1] << 8)) + ((q[2] + (q[3] << 8)) << 16),
                      (q[4] + (q[5] << 8)) + ((q[6] + (q[7] << 8)) << 16));
}

// The exact decision for all eight, out of line: few chunks need it.
template <int BITS>
__device__ __noinline__ uint2 kv_codes_exact(float4 a, float4 b, float scale, float zero) {
    const QParams g{scale, zero, __frcp_rn(scale)};
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quant_code(v[i], g, (1 << BITS) - 1);
    return pack_codes<BITS>(q);
}

// Eight codes of one chunk. fma(v, inv, magic) holds the integer nearest to v * inv (one rounding).
// up and dn are 1/scale (known to 2^-23) times 1 + 2^-22 and 1 - 2^-22, so v * up and v * dn enclose
// the exact quotient, each within 2^-21 of it (2^-22, 2^-23 and the products' roundings of
// 2^-24): where both round to one integer the quotient does too.
//   16-bit types: where they differ the quotient is a tie, and the even one of the two is taken:
//   the sum of the two rounded values, (2 magic + k + k') of spacing 2, rounds to it by itself.
//   For with v = m 2^a and scale = M 2^b (M < 2^11), a quotient other than k + 1/2 is off it by
//   |2v - (2k+1) scale| / (2v) of itself, which is at least 2^min(a+1,b) / (2v): 2^-11 where a + 1
//   < b, else 1 / (2 (k+1/2) M) > 2^-20 for k up to 255.
//   fp32: the exact decision is made (one chunk in about 100000 for 4 bits, 6500 for 8, on normal
//   data).
// Ties are not rare: one warp's pass in seven has one in bf16, where the scales often end in
// zeros (deciding them out of line took 4 % more).
// The lower clamp is implied: rint(lo/s) + rint(-lo/s) = 0.
template <typename T, int BITS>
__device__ __forceinline__ uint2 kv_codes(const float* v, const KvGrid& g) {
    constexpr int MAXQ = (1 << BITS) - 1;
    auto twice = [](float x) { return f32x2(__float_as_uint(x), __float_as_uint(x)); };
    const uint64_t up2 = twice(g.inv * (1.0f + 0x1p-22f)), dn2 = twice(g.inv * (1.0f - 0x1p-22f));
    int q[8];
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t v2 = f32x2(__float_as_uint(v[i]), __float_as_uint(v[i + 1]));
        uint64_t a = twice(kMagicInt), b = twice(kMagicInt);
        fma_f32x2(a, v2, up2);
        fma_f32x2(b, v2, dn2);
        if (sizeof(T) == 4)
            differ |= static_cast<uint32_t>(a ^ b) | static_cast<uint32_t>((a ^ b) >> 32);
        fma_f32x2(b, a, twice(1.0f));
#pragma unroll
        for (int j = 0; j < 2; ++j)
            q[i + j] = __viaddmin_s32(__float_as_int(f32x2_get(b, j)), g.to_code, MAXQ);
    }
    if (differ)
        return kv_codes_exact<BITS>(make_float4(v[0], v[1], v[2], v[3]),
                                    make_float4(v[4], v[5], v[6], v[7]), g.scale, g.zero);
    return pack_codes<BITS>(q);
}

// to_code of a zero: 2 magic + 2 k has the bits 0x4BC00000 + k, magic + zero 0x4B400000 + zero.
__device__ __forceinline__ int kv_to_code(float zero) {
    return static_cast<int>(__float_as_uint(kMagicInt + zero) - 0x97000000u);
}

// A range {minimum, -maximum} of a chunk or group, so that one minimum joins both ends; NaN if any
// value is. In the 16-bit types it is one packed register. or_if(c, o) is o where c holds.
template <typename T>
struct KvRange;
template <>
struct KvRange<__half> {
    uint32_t r;
    __device__ __forceinline__ __half2 pair() const { return *reinterpret_cast<const __half2*>(&r); }
    __device__ __forceinline__ void set(__half2 x) { r = *reinterpret_cast<const uint32_t*>(&x); }
    __device__ __forceinline__ void of(const uint4* x) {
        __half2 a, b;
        minmax_packed(x[0], a, b);
        set(__halves2half2(__hmin_nan(__low2half(a), __high2half(a)),
                          __hneg(__hmax_nan(__low2half(b), __high2half(b)))));
    }
    __device__ __forceinline__ void join(const KvRange& o) { set(__hmin2_nan(pair(), o.pair())); }
    __device__ __forceinline__ KvRange other(int mask) const {
        return {__shfl_xor_sync(0xffffffffu, r, mask)};
    }
    __device__ __forceinline__ KvRange or_if(bool c, const KvRange& o) const { return {c ? o.r : r}; }
    __device__ __forceinline__ float lo() const { return __low2float(pair()); }
    __device__ __forceinline__ float hi() const { return -__high2float(pair()); }
};
template <>
struct KvRange<__nv_bfloat16> {
    uint32_t r;
    __device__ __forceinline__ __nv_bfloat162 pair() const { return *reinterpret_cast<const __nv_bfloat162*>(&r); }
    __device__ __forceinline__ void set(__nv_bfloat162 x) { r = *reinterpret_cast<const uint32_t*>(&x); }
    __device__ __forceinline__ void of(const uint4* x) {
        __nv_bfloat162 a, b;
        minmax_packed(x[0], a, b);
        set(__halves2bfloat162(__hmin_nan(__low2bfloat16(a), __high2bfloat16(a)),
                              __hneg(__hmax_nan(__low2bfloat16(b), __high2bfloat16(b)))));
    }
    __device__ __forceinline__ void join(const KvRange& o) { set(__hmin2_nan(pair(), o.pair())); }
    __device__ __forceinline__ KvRange other(int mask) const {
        return {__shfl_xor_sync(0xffffffffu, r, mask)};
    }
    __device__ __forceinline__ KvRange or_if(bool c, const KvRange& o) const { return {c ? o.r : r}; }
    __device__ __forceinline__ float lo() const { return __low2float(pair()); }
    __device__ __forceinline__ float hi() const { return -__high2float(pair()); }
};
template <>
struct KvRange<float> {
    float mn, nmx;
    __device__ __forceinline__ void of(const uint4* x) {
        const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
        mn = __uint_as_float(w[0]);
        nmx = -mn;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            mn = min_nan(mn, __uint_as_float(w[i]));
            nmx = min_nan(nmx, -__uint_as_float(w[i]));
        }
    }
    __device__ __forceinline__ void join(const KvRange& o) {
        mn = min_nan(mn, o.mn);
        nmx = min_nan(nmx, o.nmx);
    }
    __device__ __forceinline__ KvRange other(int mask) const {
        return {__shfl_xor_sync(0xffffffffu, mn, mask), __shfl_xor_sync(0xffffffffu, nmx, mask)};
    }
    __device__ __forceinline__ KvRange or_if(bool c, const KvRange& o) const {
        return {c ? o.mn : mn, c ? o.nmx : nmx};
    }
    __device__ __forceinline__ float lo() const { return mn; }
    __device__ __forceinline__ float hi() const { return -nmx; }
};

// Quantise and write. The TPG lanes of a group join their U passes' ranges in halves: at each step a
// lane keeps one half of the passes that it still holds and hands the other half to its partner,
// so that it ends with whole ranges of ROUNDS passes, no two lanes with the same while U >= TPG,
// for U - 1 shuffles instead of U log2(TPG). Each lane computes the scalars of its own (fp64, the
// dearest part: about 100 instructions) and writes scale and zero; the lanes of a group fetch what
// they need for their codes with two shuffles per pass.
// 16384 tokens x 32 x 128, 4 bits, bf16: 60 us. On the way there: 174 us with the addresses shared
// by four passes, 129 with the exact decision out of line, 111 with the enclosing roundings, 109
// with branch-free scalars, 100 with eight passes, 96 with ties in line. Tried with four passes:
// two 144, loading a unit ahead 125, fewer registers for more warps 120.
template <typename T, int BITS, int TPG, int U>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const T* __restrict__ K,
                                                              const T* __restrict__ V, int64_t n,
                                                              int64_t k_stride, int64_t v_stride,
                                                              const int64_t* __restrict__ slots,
                                                              const KvParams p, int64_t row_step,
                                                              int wc_step) {
    constexpr int MAXQ = (1 << BITS) - 1, VEC = 8 / Vec<T>::N;
    constexpr int ROUNDS = U > TPG ? U / TPG : 1;       // passes whose scalars a lane computes
    constexpr int H = U > 1 ? U / 2 : 1;                // passes of the keys, then of the values
    pdl_wait();
    const int lane = lane_id();
    const int64_t warp0 = (static_cast<int64_t>(blockIdx.x) * kKvThreads + threadIdx.x) >> 5;
    const int64_t n_rows = U > 1 ? n : 2 * n;           // tokens, or plane rows
    int64_t row = warp0 * (32 * H) / p.wc;              // the warp's row and first chunk
    int wc0 = static_cast<int>(warp0 * (32 * H) - row * p.wc);
    while (row < n_rows) {                              // warp-uniform
        int64_t r = row;
        int wc = wc0 + lane;
        if (U == 1) {                                   // a pass may run over row ends
            while (wc >= p.wc) {
                wc -= p.wc;
                ++r;
            }
        }
        const int64_t t = U > 1 ? r : r >> 1;
        int64_t dst = -1;                               // the (first) plane row in the cache, or -1
        uint4 x[U][VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[u][i] = make_uint4(0, 0, 0, 0);
        if (U > 1 || t < n) {
            const int64_t slot = __ldg(slots + t);
            const uint4* ks = reinterpret_cast<const uint4*>(K + t * k_stride + 8 * wc);
            const uint4* vs = reinterpret_cast<const uint4*>(V + t * v_stride + 8 * wc);
            if (U == 1 && (r & 1)) ks = vs;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    x[u][i] = __ldcs((u < H ? ks : vs) + (u % H) * 32 * VEC + i);
            if (slot >= 0 && slot < p.n_slots) dst = (U == 1 && (r & 1) ? p.n_slots : 0) + slot;
            else if (slot >= 0) set_status(p.status, GPTQ_ERR_ARG);
        }
        KvRange<T> range[U];
#pragma unroll
        for (int u = 0; u < U; ++u) range[u].of(x[u]);
        int mine = 0;                                   // the lane's (first) pass
#pragma unroll
        for (int o = 1; o < TPG; o *= 2) {
            const int half = U / (2 * o);               // 0: one pass left, joined by all lanes
            const bool upper = half > 0 && (lane & o);
            if (upper) mine += half;
#pragma unroll
            for (int u = 0; u < (half > 0 ? half : 1); ++u) {
                const KvRange<T> give = range[u + half].or_if(upper, range[u]);
                range[u] = range[u].or_if(upper, range[u + half]);
                range[u].join(give.other(o));
            }
        }
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
            const float lo = range[j].lo(), hi = range[j].hi();
            // (a difference with itself is 0 for finite values only)
            const bool finite = (lo - lo) == 0.0f && (hi - hi) == 0.0f;
            const QParams grid = group_params_stream(finite ? lo : 0.0f, finite ? hi : 0.0f, MAXQ);
            const bool usable = finite && grid.scale <= 65504.0f;
            const float zero = usable ? grid.zero : 0.0f;
            const float inv = usable ? grid.inv_scale : __uint_as_float(0x7FC00000u);
            const int to_code = kv_to_code(zero);
            if (dst >= 0 && lane % TPG < U) {
                const int u = mine + j;
                const int64_t to = dst + (u < H ? 0 : p.n_slots);
                const int64_t gi = to * p.ng + (wc + 32 * (u % H)) / TPG;
                p.scales[gi] = usable ? half_bits(grid.scale) : kHalfNan;
                p.zeros[gi] = half_bits(zero);
            }
#pragma unroll
            for (int u = j; u < U; u += ROUNDS) {
                int src = 0;                            // the group's lane that has pass u
#pragma unroll
                for (int o = 1; o < TPG && U / (2 * o) > 0; o *= 2)
                    if (u & (U / (2 * o))) src += o;
                KvGrid g;
                g.inv = __shfl_sync(0xffffffffu, inv, src, TPG);
                g.to_code = __shfl_sync(0xffffffffu, to_code, src, TPG);
                if (sizeof(T) == 4) {
                    g.scale = __shfl_sync(0xffffffffu, grid.scale, src, TPG);
                    g.zero = __shfl_sync(0xffffffffu, zero, src, TPG);
                }
                float v[8];
                Vec<T>::unpack(x[u][0], v);
                if constexpr (VEC == 2) Vec<T>::unpack(x[u][1], v + 4);
                uint2 w = kv_codes<T, BITS>(v, g);
                if (!(g.inv == g.inv)) w = make_uint2(0, 0);    // no finite grid: codes 0
                if (dst >= 0) {
                    const int64_t to = dst + (u < H ? 0 : p.n_slots);
                    const int64_t at = to * p.wc + wc + 32 * (u % H);
                    if (BITS == 4) reinterpret_cast<uint32_t*>(p.codes)[at] = w.x;
                    else reinterpret_cast<uint2*>(p.codes)[at] = w;
                }
            }
        }
        row += row_step;
        wc0 += wc_step;
        if (wc0 >= p.wc) {
            wc0 -= p.wc;
            ++row;
        }
    }
}

// The largest b in [0, n_seqs] with cu[b] <= t; -1 when t < cu[0].
__device__ __forceinline__ int kv_find_seq(const int32_t* __restrict__ cu, int n_seqs, int64_t t) {
    int lo = -1, hi = n_seqs + 1;              // cu[lo] <= t < cu[hi] (virtually, at the ends)
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (__ldg(cu + mid) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Eight values of one chunk, scale * (code - zero) rounded once to T. A code's byte is placed into
// the mantissa of a constant, and two values go through one instruction:
//   fp16          1024 + code, less 1024 + zero (exact), times scale
//   else, 4 bits  fma(128 + code, scale, -scale (128 + zero)): 8 and 11 bits, so the products and
//                 their difference are exact in fp32
//   else, 8 bits  2^23 + code, less 2^23 + zero (exact), times scale (exact: 9 and 11 bits)
template <typename T, int BITS>
__device__ __forceinline__ void kv_values(uint2 w, uint16_t scale_bits, uint16_t zero_bits, T* at,
                                          int wide) {
    const uint32_t even = w.x & 0x0F0F0F0Fu, odd = (w.x >> 4) & 0x0F0F0F0Fu;     // for 4 bits
    const __half hs = __ushort_as_half(scale_bits), hz = __ushort_as_half(zero_bits);
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 s2 = __half2half2(hs);
        const __half2 z2 = __half2half2(__hadd(hz, __ushort_as_half(0x6400)));
        const uint32_t lo = BITS == 4 ? __byte_perm(even, odd, 0x5140) : w.x;
        const uint32_t hi = BITS == 4 ? __byte_perm(even, odd, 0x7362) : w.y;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __byte_perm(i < 2 ? lo : hi, 0x64646464u, i & 1 ? 0x4342 : 0x4140);
            const __half2 y = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&x), z2), s2);
            o[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
        *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
        auto twice = [](float x) { return f32x2(__float_as_uint(x), __float_as_uint(x)); };
        const float scale = __half2float(hs), zero = __half2float(hz);
        const uint64_t s2 = twice(scale);
        const uint64_t z2 = twice(BITS == 4 ? -scale * (128.0f + zero) : -(8388608.0f + zero));
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            uint64_t y = z2;
            if (BITS == 4) {
                const int sel = 0x7044 + (i / 2 << 8);
                fma_f32x2(y, f32x2(__byte_perm(even, 0x43000000u, sel),
                                   __byte_perm(odd, 0x43000000u, sel)), s2);
            } else {
                const uint32_t word = i < 4 ? w.x : w.y;
                const int b = i & 2;           // the pair's first byte
                fma_f32x2(y, f32x2(__byte_perm(word, 0x4B000000u, 0x7440 + b),
                                   __byte_perm(word, 0x4B000000u, 0x7441 + b)), twice(1.0f));
                const uint64_t d = y;
                y = 0;
                fma_f32x2(y, d, s2);
            }
            v[i] = f32x2_get(y, 0);
            v[i + 1] = f32x2_get(y, 1);
        }
        kv_store8(at, v, wide);
    }
}

// Read back. A CTA takes consecutive tokens: 1 << log_parts warps share each, and a warp has every
// `apart`-th one, `rows` (1 to 32) of them. Lane i finds the warp's token i's sequence, page and
// slot, and the warp then runs over the tokens' chunks, U passes of loads at a time.
// The order of the writes decides the rest: 16384 x 32 x 128, 4 bits, bf16, took 70 us with four
// passes and 32 or fewer consecutive tokens per warp, 64 with eight passes, 60 with all warps
// writing side by side. (With 9 instructions per value instead of 7 it took the same.)
template <typename T, int BITS, int U>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvParams p, int page_size,
                                                             int64_t n_pages,
                                                             const int32_t* __restrict__ table,
                                                             int n_seqs, int max_pages,
                                                             const int32_t* __restrict__ cu,
                                                             int64_t total, int rows, int log_parts,
                                                             T* __restrict__ K, T* __restrict__ V,
                                                             int wide) {
    constexpr int H = U > 1 ? U / 2 : 1;       // passes of the keys, then of the values
    constexpr int64_t kNobody = -2, kMissing = -1;
    pdl_wait();
    const int lane = lane_id();
    const int parts = 1 << log_parts;                        // warps of a token
    const int apart = (kKvThreads / 32) >> log_parts;        // tokens between a warp's
    const int first_chunk = (warp_id() & (parts - 1)) * 32 * H;
    const int64_t step = static_cast<int64_t>(gridDim.x) * apart * rows;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * apart * rows + (warp_id() >> log_parts);
         t0 < total; t0 += step) {
        const int64_t t = t0 + lane * apart;                 // the token that the lane looks up
        int64_t mine = kNobody;
        if (lane < rows && t < total) {
            const int b = kv_find_seq(cu, n_seqs, t);
            if (b >= 0 && b < n_seqs) {        // else a row of no sequence: left as it was
                const int64_t pos = t - __ldg(cu + b);
                mine = kMissing;
                if (pos >= 0) {
                    const unsigned pi = static_cast<unsigned>(pos) / static_cast<unsigned>(page_size);
                    if (pi < static_cast<unsigned>(max_pages)) {
                        const int64_t page = __ldg(table + static_cast<int64_t>(b) * max_pages + pi);
                        if (page >= 0 && page < n_pages)
                            mine = page * page_size + (pos - static_cast<int64_t>(pi) * page_size);
                    }
                }
                if (mine == kMissing) set_status(p.status, GPTQ_ERR_ARG);
            }
        }
        const int n_tok =
            static_cast<int>(min(static_cast<int64_t>(rows), (total - t0 + apart - 1) >> (2 - log_parts)));
        const int n_rows = U > 1 ? n_tok : 2 * n_tok;   // tokens, or plane rows
        int r = 0, wc = first_chunk + lane;    // the lane's row and chunk
        for (int base = first_chunk; base < n_rows * p.wc; base += parts * 32 * H) {
            while (wc >= p.wc) {
                wc -= p.wc;
                ++r;
            }
            const int tok = U > 1 ? r : r >> 1;
            const int64_t slot = __shfl_sync(0xffffffffu, mine, tok & 31);
            if (r < n_rows && slot != kNobody) {
                uint2 w[U];
                uint16_t sb[U], zb[U];
                const int64_t row = (U == 1 && (r & 1) ? p.n_slots : 0) + slot;
                const int64_t c0 = row * p.wc + wc, g0 = row * p.ng + (wc >> p.tpg_shift);
                const int g_step = 32 >> p.tpg_shift;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + (u < H ? 0 : p.n_slots * p.wc) + 32 * (u % H);
                    const int64_t g = g0 + (u < H ? 0 : p.n_slots * p.ng) + (u % H) * g_step;
                    w[u] = make_uint2(0, 0);
                    sb[u] = zb[u] = 0;
                    if (slot >= 0) {
                        if (BITS == 4) w[u].x = __ldg(reinterpret_cast<const uint32_t*>(p.codes) + c);
                        else w[u] = __ldg(reinterpret_cast<const uint2*>(p.codes) + c);
                        sb[u] = __ldg(p.scales + g);
                        zb[u] = __ldg(p.zeros + g);
                    }
                }
                const int64_t out = (t0 + tok * apart) * p.width + 8 * wc;
                T* first = (U == 1 && (r & 1) ? V : K) + out;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    kv_values<T, BITS>(w[u], sb[u], zb[u], (u < H ? first : V + out) + 256 * (u % H),
                                       wide);
                }
            }
            wc += parts * 32 * H;
        }
        __syncwarp();
    }
}

template <typename T, int BITS, int TPG, int U>
static gptq_status kv_write_go(const T* K, const T* V, int64_t n, int64_t ks, int64_t vs,
                               const int64_t* slots, const KvParams& p, cudaStream_t s) {
    constexpr int64_t kChunks = 32 * (U > 1 ? U / 2 : 1) * (kKvThreads / 32);   // of a CTA's rows
    const int64_t want = ((U > 1 ? n : 2 * n) * p.wc + kChunks - 1) / kChunks;
    const int grid = static_cast<int>(std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * 16));
    const int64_t stride = grid * kChunks;
    GPTQ_CUDA_TRY(launch_pdl(kv_write_kernel<T, BITS, TPG, U>, dim3(grid), dim3(kKvThreads), 0, s, K, V,
                             n, ks, vs, slots, p, stride / p.wc, static_cast<int>(stride % p.wc)));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
}

template <typename T, int BITS, int U>
static gptq_status kv_write_group(const T* K, const T* V, int64_t n, int64_t ks, int64_t vs,
                                  const int64_t* slots, const KvParams& p, cudaStream_t s) {
    switch (p.tpg_shift) {
        case 1: return kv_write_go<T, BITS, 2, U>(K, V, n, ks, vs, slots, p, s);
        case 2: return kv_write_go<T, BITS, 4, U>(K, V, n, ks, vs, slots, p, s);
        case 3: return kv_write_go<T, BITS, 8, U>(K, V, n, ks, vs, slots, p, s);
        case 4: return kv_write_go<T, BITS, 16, U>(K, V, n, ks, vs, slots, p, s);
        default: return kv_write_go<T, BITS, 32, U>(K, V, n, ks, vs, slots, p, s);
    }
}

template <typename T>
static gptq_status kv_write_launch(const void* K, const void* V, int64_t n, int64_t ks, int64_t vs,
                                   const int64_t* slots, int bits, const KvParams& p,
                                   cudaStream_t s) {
    const T* k = static_cast<const T*>(K);
    const T* v = static_cast<const T*>(V);
#define KV_WRITE(U)                                                             \
    (bits == 4 ? kv_write_group<T, 4, U>(k, v, n, ks, vs, slots, p, s) \
               : kv_write_group<T, 8, U>(k, v, n, ks, vs, slots, p, s))
    // 16384 x 32 x 128 in bf16 takes 62 us with eight passes, 72 with four, 105 with two (groups of
    // 16: 85, 88, 103); a few tokens take the same with any.
    if (p.wc % 128 == 0) return KV_WRITE(8);
    if (p.wc % 64 == 0) return KV_WRITE(4);
    if (p.wc % 32 == 0) return KV_WRITE(2);
    return KV_WRITE(1);
#undef KV_WRITE
}

static bool kv_aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

template <typename T>
static gptq_status kv_read_launch(const KvParams& p, int page_size, int64_t n_pages,
                                  const int32_t* table, int n_seqs, int max_pages,
                                  const int32_t* cu, int64_t total, void* K, void* V, int bits,
                                  cudaStream_t s) {
    // Up to four warps take a token's passes in turn, and a warp takes as many tokens as make 8 KB,
    // sharing the search, so that all CTAs together write one stretch of memory after the other.
    // 16384 x 32 x 128, 8 bits: 66 us with one token per warp, 67 with two, 83 with 32 (65 and 80
    // with a warp per token); 131072 tokens x 4 x 128, 1000 sequences: 81, 66, 79, with four 64.
    int log_parts = 0;
    while (log_parts < 2 && (128 << log_parts) < p.wc) ++log_parts;
    const int64_t bytes = 2 * static_cast<int64_t>(p.width) * static_cast<int64_t>(sizeof(T));
    const int64_t warps = static_cast<int64_t>(num_sms()) * 32;
    int rows = 1;
    while (rows < 32 && 2 * rows * bytes <= 8192 && 2 * rows * warps <= total << log_parts) rows *= 2;
    const int64_t per_cta = rows * ((kKvThreads / 32) >> log_parts);
    const int64_t want = (total + per_cta - 1) / per_cta;
    const int grid = static_cast<int>(std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * 64));
    T* k = static_cast<T*>(K);
    T* v = static_cast<T*>(V);
#define KV_READ(U) (bits == 4 ? kv_read_kernel<T, 4, U> : kv_read_kernel<T, 8, U>)
    // eight passes at a time while warps are scarce (512 tokens x 32 x 128, 4 bits: 4.2 us, 5.2 with
    // four), else four (131072 x 8 x 128, 4 bits: 114 us, 118 with eight, 125 with two)
    const bool few = (total << log_parts) <= 2 * warps;
    auto* kernel = p.wc % 128 == 0 && few ? KV_READ(8)
                   : p.wc % 64 == 0       ? KV_READ(4)
                   : p.wc % 32 == 0       ? KV_READ(2)
                                          : KV_READ(1);
#undef KV_READ
    GPTQ_CUDA_TRY(launch_pdl(kernel, dim3(grid), dim3(kKvThreads), 0, s, p, page_size, n_pages, table,
                             n_seqs, max_pages, cu, total, rows, log_parts, k, v,
                             kv_aligned(K, 32) && kv_aligned(V, 32) ? 1 : 0));
    GPTQ_LAUNCHED();
    return GPTQ_OK;
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
    p->tpg_shift = 1;
    while ((16 << (p->tpg_shift - 1)) < group_size) ++p->tpg_shift;
    p->codes = static_cast<uint8_t*>(const_cast<void*>(codes));
    p->scales = static_cast<uint16_t*>(const_cast<void*>(scales));
    p->zeros = static_cast<uint16_t*>(const_cast<void*>(zeros));
    p->status = status;
    return GPTQ_OK;
}

// Whether [x, x + bytes) shares memory with one of the cache's arrays.
static bool kv_in_cache(const KvParams& p, int bits, const void* x, int64_t bytes) {
    const int64_t rows = 2 * p.n_slots;
    return overlap(x, bytes, p.codes, rows * p.width * bits / 8) ||
           overlap(x, bytes, p.scales, rows * p.ng * 2) || overlap(x, bytes, p.zeros, rows * p.ng * 2);
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
    // tokens are read while others' codes are written
    auto bytes = [&](int64_t stride) {
        return gq::range_bytes((n_tokens - 1) * stride + p.width, dtype == GPTQ_DTYPE_F32 ? 4 : 2);
    };
    if (gq::kv_in_cache(p, bits, K, bytes(k_stride)) || gq::kv_in_cache(p, bits, V, bytes(v_stride)) ||
        gq::kv_in_cache(p, bits, slots, 8 * n_tokens))
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
    const int64_t out = gq::range_bytes(total * p.width, dtype == GPTQ_DTYPE_F32 ? 4 : 2);
    if (gq::overlap(K, out, V, out) || gq::kv_in_cache(p, bits, K, out) ||
        gq::kv_in_cache(p, bits, V, out))
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
