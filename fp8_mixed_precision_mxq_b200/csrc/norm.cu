// norm.cu -- the norms before and after a transformer block, fused with the block's gate,
// the residual sum and the next linear's activation quantizer.
//
// Per row of K channels (x the residual stream, y the block's output):
//   u = post(y)                          post: none, LayerNorm or RMSNorm
//   z = x + gate * u                     rounded once to the stream's type
//   n = norm(z)                          LayerNorm or RMSNorm of the rounded z
//   h = bf16(n * (1 + scale) + shift)    as bf16, or as MX codes and tiled E8M0 scales
// with LayerNorm(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps), RMSNorm(v) = v /
// sqrt(mean(v^2) + eps), each times its weight plus its bias where given.  Everything between
// the loads and the two roundings is binary32, the statistics taken in two passes over the
// row in registers (first the mean, then the centered squares) and the mean of an fp32 row far
// from zero in a second round, so a large common offset costs no digits and a constant row
// normalizes to zeros.
//
// A CTA holds its rows in registers: x and y are read once and z and h written once, which is
// all the traffic there is; HBM bounds it.  The per-channel vectors (gate, scale, shift, weights)
// are shared by all rows of a group and come from L1.
#include <cuda_bf16.h>

#include <algorithm>

#include "mx_elem.cuh"
#include "mxq_internal.h"
#include "ptx.cuh"

namespace mxq {

namespace {

constexpr int kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;

// Registers a thread may take, so that many rows are under way on an SM.  Measured at 5120 channels
// only (32760 rows; gate, scale and shift in fp32): one row of two chunks a thread at 48 registers
// 240 us (bf16 out), at 56 269, at 40 273; two rows at 64 registers 284, but with E4M3 out 559 us
// (75600 rows) against 591; an fp32 stream two rows at 80 registers 317 us, one row at 64 374.
// The budgets do not hold everything: with one or two rows of two chunks only the kernels of a
// bf16 stream with MX out spill (92-136 bytes a thread), but with four rows of one chunk a bf16
// stream spills 80-144 bytes, and with four chunks a thread every kernel 92-364.
constexpr int norm_regs(bool f32, int c, int r, bool early)
{
    return early ? 128 : c * r < 4 ? (f32 ? 64 : 48) : f32 && c < 4 ? 80 : 64;
}


struct NormParams {
    const void* x;
    const void* y;
    const void* gate;
    const void* scale;
    const void* shift;
    const void* weight;
    const void* bias;
    const void* post_weight;
    const void* post_bias;
    void* z;
    void* out;    // h in bf16, or the codes
    uint8_t* sf;  // tiled scales (quantized h)
    int64_t rows;
    int64_t rows_pad;    // rows of the scale layout
    int64_t row_blocks;  // CTAs that have rows; the rest write the layout's padding
    int e4m3;            // a quantized h's format
    uint32_t K;
    uint32_t rows_per_group;
    uint32_t atoms_k;
    float eps;
    float inv_k;
    int norm, post;  // MXQ_NORM_*
};

// A thread's eight channels of a 256-channel span: four at 4 * lane and four at 128 + 4 * lane, so
// that a warp's every load and store of fp32 or bf16 values is one contiguous run (eight
// neighbouring channels a thread would spread an fp32 load over twice its cache lines, which the
// L1 pipe felt: 70 % busy).  w: the values as they lie in memory.
template <bool kF32>
struct Raw8 {
    uint4 w[kF32 ? 2 : 1];
};

// at: the channels of the two fours.
struct At {
    uint32_t a, b;
};

template <bool kF32, class T>
__device__ __forceinline__ T* at4(T* p, size_t i)
{
    return p + i * (kF32 ? 4 : 2);
}

// Channel vectors: shared by the rows, kept in L1.
template <bool kF32>
__device__ __forceinline__ Raw8<kF32> load_vec8(const void* p, size_t base, const At& at)
{
    const uint8_t* q = at4<kF32>(static_cast<const uint8_t*>(p), base);
    Raw8<kF32> r;
    if constexpr (kF32) {
        r.w[0] = __ldg(reinterpret_cast<const uint4*>(at4<true>(q, at.a)));
        r.w[1] = __ldg(reinterpret_cast<const uint4*>(at4<true>(q, at.b)));
    } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(at4<false>(q, at.a)));
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(at4<false>(q, at.b)));
        r.w[0] = make_uint4(a.x, a.y, b.x, b.y);
    }
    return r;
}

// The rows themselves are read once: streaming loads, which leave L1 to the vectors.
template <bool kF32>
__device__ __forceinline__ Raw8<kF32> load_row8(const void* p, size_t base, const At& at)
{
    const uint8_t* q = at4<kF32>(static_cast<const uint8_t*>(p), base);
    Raw8<kF32> r;
    if constexpr (kF32) {
        r.w[0] = __ldcs(reinterpret_cast<const uint4*>(at4<true>(q, at.a)));
        r.w[1] = __ldcs(reinterpret_cast<const uint4*>(at4<true>(q, at.b)));
    } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(at4<false>(q, at.a)));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(at4<false>(q, at.b)));
        r.w[0] = make_uint4(a.x, a.y, b.x, b.y);
    }
    return r;
}

// live_a, live_b: whether the fours lie inside the row.
template <bool kF32>
__device__ __forceinline__ void store_row8(void* p, size_t base, const At& at, bool live_a, bool live_b,
                                           const Raw8<kF32>& r)
{
    uint8_t* q = at4<kF32>(static_cast<uint8_t*>(p), base);
    if constexpr (kF32) {
        if (live_a) *reinterpret_cast<uint4*>(at4<true>(q, at.a)) = r.w[0];
        if (live_b) *reinterpret_cast<uint4*>(at4<true>(q, at.b)) = r.w[1];
    } else {
        if (live_a) *reinterpret_cast<uint2*>(at4<false>(q, at.a)) = make_uint2(r.w[0].x, r.w[0].y);
        if (live_b) *reinterpret_cast<uint2*>(at4<false>(q, at.b)) = make_uint2(r.w[0].z, r.w[0].w);
    }
}

// Values past the row's end are zeros.
template <bool kF32>
__device__ __forceinline__ void zero_dead(Raw8<kF32>& r, bool live_a, bool live_b)
{
    const uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (kF32) {
        if (!live_a) r.w[0] = o;
        if (!live_b) r.w[1] = o;
    } else {
        if (!live_a) r.w[0].x = r.w[0].y = 0u;
        if (!live_b) r.w[0].z = r.w[0].w = 0u;
    }
}

template <bool kF32>
__device__ __forceinline__ void widen8(const Raw8<kF32>& r, float2 (&v)[4])
{
    if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[2 * i] = make_float2(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
            v[2 * i + 1] = make_float2(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
        }
    } else {
        v[0] = make_float2(lo_f(r.w[0].x), hi_f(r.w[0].x));
        v[1] = make_float2(lo_f(r.w[0].y), hi_f(r.w[0].y));
        v[2] = make_float2(lo_f(r.w[0].z), hi_f(r.w[0].z));
        v[3] = make_float2(lo_f(r.w[0].w), hi_f(r.w[0].w));
    }
}

// Stops the compiler from holding a packed chunk's widened values from one pass to the next.
template <bool kF32>
__device__ __forceinline__ void keep_packed(Raw8<kF32>& r)
{
    if constexpr (!kF32) asm volatile("" : "+r"(r.w[0].x), "+r"(r.w[0].y), "+r"(r.w[0].z), "+r"(r.w[0].w));
}

__device__ __forceinline__ uint4 pack8(const float2 (&v)[4])
{
    return make_uint4(bf16x2_bits(v[0].x, v[0].y), bf16x2_bits(v[1].x, v[1].y), bf16x2_bits(v[2].x, v[2].y),
                      bf16x2_bits(v[3].x, v[3].y));
}

template <bool kF32>
__device__ __forceinline__ void narrow8(const float2 (&v)[4], Raw8<kF32>& r)
{
    if constexpr (kF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = make_uint4(__float_as_uint(v[2 * i].x), __float_as_uint(v[2 * i].y), __float_as_uint(v[2 * i + 1].x),
                                __float_as_uint(v[2 * i + 1].y));
    } else {
        r.w[0] = pack8(v);
    }
}

// Sums over the CTA, the same values in every thread.  `red` is used by this call only.
template <int R>
__device__ __forceinline__ void block_sum(float (&v)[R], float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xFFFFFFFFu, v[r], o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) red[r * kMaxWarps + (threadIdx.x >> 5)] = v[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = lane < warps ? red[r * kMaxWarps + lane] : 0.0f;
#pragma unroll
        for (int o = kMaxWarps / 2; o > 0; o >>= 1) v[r] += __shfl_xor_sync(0xFFFFFFFFu, v[r], o);
    }
}

// A mean beyond this many standard deviations is taken again (row_stats).
constexpr float kFarMean = 16.0f;

// -mean (0 for RMSNorm) and 1 / sqrt(variance + eps) of the CTA's rows.  Channels past K (`live`
// false; with kFull there are none) are held as zeros and left out of the centered squares.
// load(r, j, t) gives chunk j of row r.
// An error of the mean is multiplied by 1 / sqrt(variance + eps), a thousandfold in a constant row,
// which has to come out as zeros.  kBf16 (the values are): values of like size, up to 2^15 of them of
// eight bits, sum exactly, and one residual step after the product with the rounded 1 / K (Markstein's
// division) gives the quotient, rounded once; a constant row's mean is exact.  Otherwise the sum is
// rounded as well; so where the mean is far (rare; all threads agree, and row by row, so that a row's
// result does not depend on its neighbours) the centered values, which are small, are summed too and
// their mean is added: -mean is then neg_mean + lo[r] to about twice binary32's digits.  (For the fp32
// stream this costs 1 to 3 %; for bf16 it would cost 10 % at 5120 channels, in spills.)
template <bool kBf16, int R, int C, bool kFull, class F>
__device__ __forceinline__ void row_stats(F load, const bool (&live)[C][2], int kind, uint32_t K, float inv_k,
                                          float eps, float* red, float (&neg_mean)[R], float (&lo)[R],
                                          float (&rstd)[R])
{
#pragma unroll
    for (int r = 0; r < R; ++r) lo[r] = 0.0f;
    float2 t[4];
    if (kind == MXQ_NORM_LAYER) {
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                load(r, j, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) a = __fadd2_rn(a, t[i]);
            }
            s[r] = a.x + a.y;
        }
        block_sum<R>(s, red);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            neg_mean[r] = -(s[r] * inv_k);
            if constexpr (kBf16) neg_mean[r] = fmaf(-fmaf(neg_mean[r], static_cast<float>(K), s[r]), inv_k, neg_mean[r]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                load(r, j, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float m = kFull || live[j][i / 2] ? neg_mean[r] : 0.0f;
                    const float2 d = __fadd2_rn(t[i], make_float2(m, m));
                    q = __ffma2_rn(d, d, q);
                }
            }
            rstd[r] = q.x + q.y;
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            neg_mean[r] = 0.0f;
            float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                load(r, j, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) q = __ffma2_rn(t[i], t[i], q);
            }
            rstd[r] = q.x + q.y;
        }
    }
    block_sum<R>(rstd, red + R * kMaxWarps);
    if (!kBf16 && kind == MXQ_NORM_LAYER) {
        bool far[R], any = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            far[r] = neg_mean[r] * neg_mean[r] > kFarMean * kFarMean * inv_k * rstd[r];
            any = any || far[r];
        }
        if (any) {
            const float k = static_cast<float>(K);
            float s[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    load(r, j, t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float m = kFull || live[j][i / 2] ? neg_mean[r] : 0.0f;
                        a = __fadd2_rn(a, __fadd2_rn(t[i], make_float2(m, m)));
                    }
                }
                s[r] = a.x + a.y;
            }
            block_sum<R>(s, red);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float d = __fdiv_rn(s[r], k), m = neg_mean[r] - d;
                if (far[r]) {
                    lo[r] = (neg_mean[r] - m) - d;  // what the sum rounded off
                    neg_mean[r] = m;
                }
                float2 q = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    load(r, j, t);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float mi = kFull || live[j][i / 2] ? neg_mean[r] : 0.0f;
                        const float2 c = __fadd2_rn(t[i], make_float2(mi, mi));
                        q = __ffma2_rn(c, c, q);
                    }
                }
                s[r] = q.x + q.y;
            }
            block_sum<R>(s, red + R * kMaxWarps);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (far[r]) rstd[r] = fmaxf(fmaf(-k * lo[r], lo[r], s[r]), 0.0f);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) rstd[r] = __frsqrt_rn(rstd[r] * inv_k + eps);
}

struct Mul {
    __device__ float2 operator()(float2 a, float2 t) const { return __fmul2_rn(a, t); }
};
struct Add {
    __device__ float2 operator()(float2 a, float2 t) const { return __fadd2_rn(a, t); }
};
struct MulOnePlus {
    __device__ float2 operator()(float2 a, float2 t) const
    {
        return __fmul2_rn(a, __fadd2_rn(t, make_float2(1.0f, 1.0f)));
    }
};

// v = f(v, vector) on the threads' chunks of all rows, the vector from memory (`base`: of its
// first channel) or already in registers.
template <bool kVF32, int R, int C, class F>
__device__ __forceinline__ void apply_vec(float2 (&v)[R][C][4], const void* from, size_t base, const At (&at)[C], F f)
{
#pragma unroll
    for (int j = 0; j < C; ++j) {
        float2 t[4];
        widen8(load_vec8<kVF32>(from, base, at[j]), t);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][j][i] = f(v[r][j][i], t[i]);
    }
}

template <bool kVF32, int R, int C, class F>
__device__ __forceinline__ void apply_vec(float2 (&v)[R][C][4], const Raw8<kVF32> (&from)[C], F f)
{
#pragma unroll
    for (int j = 0; j < C; ++j) {
        float2 t[4];
        widen8(from[j], t);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[r][j][i] = f(v[r][j][i], t[i]);
    }
}

// v = (v + neg_mean + lo) * rstd.
template <int R, int C>
__device__ __forceinline__ void normalize(float2 (&v)[R][C][4], const float (&neg_mean)[R], const float (&lo)[R],
                                          const float (&rstd)[R])
{
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float at0 = lo[r] == 0.0f ? 0.0f : lo[r] * rstd[r];
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[r][j][i] = __ffma2_rn(__fadd2_rn(v[r][j][i], make_float2(neg_mean[r], neg_mean[r])),
                                        make_float2(rstd[r], rstd[r]), make_float2(at0, at0));
    }
}

// Writes one chunk of h: in bf16, or as MX codes and scale bytes.  c: its first channel.
template <bool kQuant>
__device__ __forceinline__ void emit(const NormParams& p, int64_t row, size_t base, uint32_t c, const At& at, bool live_a,
                                     bool live_b, const float2 (&v)[4])
{
    Raw8<false> h;
    narrow8(v, h);
    if constexpr (!kQuant) {
        store_row8(p.out, base, at, live_a, live_b, h);
    } else {
        // eight lanes' fours are one MX block (two, a and b): the activation quantizer's
        // arithmetic on the bf16 h (scale from the abs-max's exponent field, codes rounded
        // to nearest even with saturation, zero codes in a non-finite block)
        const uint32_t ma = absmax_bf16x2(h.w[0].x, h.w[0].y), mb = absmax_bf16x2(h.w[0].z, h.w[0].w);
        uint32_t m = absmax_bf16x2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));  // a low, b high
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const uint32_t emax = p.e4m3 ? 8u : 2u;
        const uint32_t ea = (m >> 7) & 255u, eb = (m >> 23) & 255u;
        uint32_t sa = max(ea, emax) - emax, sb = max(eb, emax) - emax;
        const float ia = __uint_as_float((254u - sa) << 23), ib = __uint_as_float((254u - sb) << 23);  // 2^(127 - s)
        float2 q[4];
        widen8(h, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __fmul2_rn(q[i], i < 2 ? make_float2(ia, ia) : make_float2(ib, ib));
        const bool nan_a = ea == 255u, nan_b = eb == 255u;
        const bool odd = __any_sync(0xFFFFFFFFu, nan_a || nan_b);  // a non-finite block in the warp: rare
        if (nan_a) sa = 255u;
        if (nan_b) sb = 255u;
        uint8_t* codes = static_cast<uint8_t*>(p.out);
        if (p.e4m3) {
            uint32_t ca = cvt_e4m3x2(q[0].x, q[0].y) | (cvt_e4m3x2(q[1].x, q[1].y) << 16);
            uint32_t cb = cvt_e4m3x2(q[2].x, q[2].y) | (cvt_e4m3x2(q[3].x, q[3].y) << 16);
            if (odd) {
                if (nan_a) ca = 0u;
                if (nan_b) cb = 0u;
            }
            if (live_a) *reinterpret_cast<uint32_t*>(codes + base + at.a) = ca;
            if (live_b) *reinterpret_cast<uint32_t*>(codes + base + at.b) = cb;
        } else {
            const float f[8] = {q[0].x, q[0].y, q[1].x, q[1].y, q[2].x, q[2].y, q[3].x, q[3].y};
            uint32_t e = cvt_e2m1x8(f);
            if (odd) {
                if (nan_a) e &= 0xFFFF0000u;
                if (nan_b) e &= 0x0000FFFFu;
            }
            if (live_a) *reinterpret_cast<uint16_t*>(codes + (base + at.a) / 2) = static_cast<uint16_t>(e);
            if (live_b) *reinterpret_cast<uint16_t*>(codes + (base + at.b) / 2) = static_cast<uint16_t>(e >> 16);
        }
        if ((threadIdx.x & 7u) == 0) {
            // the blocks' scale bytes; k-blocks past K in the last atom are 0
            uint8_t* sf = p.sf + sf_word(row, 0, p.atoms_k) + (c / 32u & 3u);
            if (c < p.atoms_k * 128u) sf[(c / 128u) * 512u] = live_a ? static_cast<uint8_t>(sa) : uint8_t(0);
            if (c + 128u < p.atoms_k * 128u) sf[(c / 128u) * 512u + 512u] = live_b ? static_cast<uint8_t>(sb) : uint8_t(0);
        }
    }
}

// A CTA takes up to R rows of one group (of groups shorter than R rows, fewer: the rest of its work
// is thrown away; vectors of one row each, 32760 x 2048, 375 us against 107 with one group).  kF32:
// the residual stream x, z is fp32 (else bf16); kVF32: so are the channel vectors.  kQuant: h
// leaves as MX codes (else bf16).  C: chunks of 8 channels per thread and row; chunk j of warp w is
// its lanes' part of span j * warps + w, whose MX blocks lie in eight lanes each.  kFull: a row has
// exactly C * warps spans (else some channels are past its end).  kEarly: the last step's vectors
// are fetched with the rows.
// What keeps the kernel from the memory's rate is its own work, so: R rows share each vector's
// loads and each barrier; arithmetic runs on packed fp32 pairs; a bf16 z is held packed between
// the passes over it, which leaves registers for more rows on an SM; and each optional vector is
// one branch around a loop over all the thread's values (tested chunk by chunk the options
// became predicates, and a launch issued every option's instructions: 41 an element).  Many small
// CTAs hide each other's barriers: persistent CTAs, with the next row prefetched into shared
// memory, into L2 or into registers, all measured 20 to 60 % slower.
// Measured (share of the copy rate): 32760 x 5120 with gate, scale, shift in fp32, bf16 out 229-248 us
// (84-91 %), of an fp32 stream 309 us; 75600 x 5120 with E4M3 out 540-610 us (78-69 %; the slower end
// with the GPU idle between calls or after long runs).
template <bool kF32, bool kVF32, bool kQuant, int C, int R, bool kFull, bool kEarly>
__global__ void __maxnreg__(norm_regs(kF32, C, R, kEarly)) norm_residual_kernel(const NormParams p)
{
    __shared__ float red[4 * R * kMaxWarps];
    grid_launch_dependents();  // a few-row GEMM behind it sets up meanwhile
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t per_group = (p.rows_per_group + R - 1) / R;  // CTAs a group
    const uint32_t group = blockIdx.x / per_group;
    const int64_t row0 = static_cast<int64_t>(group) * p.rows_per_group + (blockIdx.x - group * per_group) * R;
    const int64_t group_end = min(static_cast<int64_t>(group + 1) * p.rows_per_group, p.rows);
    if (row0 >= group_end) {
        // CTAs past the rows take the rows of the scale layout's padding
        const int64_t row = p.rows + (static_cast<int64_t>(blockIdx.x) - p.row_blocks);
        if (kQuant && row >= p.rows && row < p.rows_pad)
            for (uint32_t a = threadIdx.x; a < p.atoms_k; a += blockDim.x)
                *reinterpret_cast<uint32_t*>(p.sf + sf_word(row, a, p.atoms_k)) = 0u;
        return;
    }
    const int rows = static_cast<int>(min(static_cast<int64_t>(R), group_end - row0));
    const size_t gbase = static_cast<size_t>(group) * p.K;
    using Vec = Raw8<kVF32>;

    // Channels past the end load the row's first ones instead and their values are zeroed.  Rows past
    // the CTA's last load that one; they store nothing.
    const uint32_t c0 = (threadIdx.x >> 5) * 256u + lane * 4u, step = blockDim.x * 8u;
    bool live[C][2];
    At at[C];
    size_t base[R];
    Raw8<kF32> z[R][C];  // x, then z
    Raw8<false> y[R][C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t c = c0 + j * step;
        live[j][0] = kFull || c < p.K;
        live[j][1] = kFull || c + 128u < p.K;
        at[j].a = live[j][0] ? c : 0u;
        at[j].b = live[j][1] ? c + 128u : 0u;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        base[r] = static_cast<size_t>(row0 + min(r, rows - 1)) * p.K;
#pragma unroll
        for (int j = 0; j < C; ++j) z[r][j] = load_row8<kF32>(p.x, base[r], at[j]);
    }
    if (p.y) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < C; ++j) y[r][j] = load_row8<false>(p.y, base[r], at[j]);
    }
    [[maybe_unused]] Vec w_r[C], b_r[C], s_r[C], t_r[C];
    if constexpr (kEarly) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (p.weight) w_r[j] = load_vec8<kVF32>(p.weight, 0, at[j]);
            if (p.bias) b_r[j] = load_vec8<kVF32>(p.bias, 0, at[j]);
            if (p.scale) s_r[j] = load_vec8<kVF32>(p.scale, gbase, at[j]);
            if (p.shift) t_r[j] = load_vec8<kVF32>(p.shift, gbase, at[j]);
        }
    }

    float neg_mean[R], lo[R], rstd[R];
    if (p.y) {
        if (p.post != MXQ_NORM_NONE) {
            if constexpr (!kFull) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int j = 0; j < C; ++j)
                        zero_dead(y[r][j], live[j][0], live[j][1]);
            }
            row_stats<true, R, C, kFull>([&](int r, int j, float2(&t)[4]) { keep_packed(y[r][j]); widen8(y[r][j], t); }, live,
                                   p.post, p.K, p.inv_k, p.eps, red + 2 * R * kMaxWarps, neg_mean, lo, rstd);
        }
        // z = x + gate * u, chunk by chunk
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float2 u[R][1][4];
            const At a1[1] = {at[j]};
#pragma unroll
            for (int r = 0; r < R; ++r) widen8(y[r][j], u[r][0]);
            if (p.post != MXQ_NORM_NONE) {
                normalize(u, neg_mean, lo, rstd);
                if (p.post_weight) apply_vec<kVF32>(u, p.post_weight, 0, a1, Mul());
                if (p.post_bias) apply_vec<kVF32>(u, p.post_bias, 0, a1, Add());
            }
            if (p.gate) {
                float2 t[4], xv[4];
                widen8(load_vec8<kVF32>(p.gate, gbase, at[j]), t);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    widen8(z[r][j], xv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[r][0][i] = __ffma2_rn(t[i], u[r][0][i], xv[i]);
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 xv[4];
                    widen8(z[r][j], xv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) u[r][0][i] = __fadd2_rn(u[r][0][i], xv[i]);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                narrow8(u[r][0], z[r][j]);  // rounded to the stream's type; the norm sees this value
                if (r < rows) store_row8(p.z, base[r], at[j], live[j][0], live[j][1], z[r][j]);
            }
        }
    }
    if constexpr (!kFull) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < C; ++j)
                zero_dead(z[r][j], live[j][0], live[j][1]);
    }
    row_stats<!kF32, R, C, kFull>([&](int r, int j, float2(&t)[4]) { keep_packed(z[r][j]); widen8(z[r][j], t); }, live, p.norm,
                           p.K, p.inv_k, p.eps, red, neg_mean, lo, rstd);
    float2 v[R][C][4];  // h
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < C; ++j) {
            keep_packed(z[r][j]);
            widen8(z[r][j], v[r][j]);
        }
    normalize(v, neg_mean, lo, rstd);
    if constexpr (kEarly) {
        if (p.weight) apply_vec<kVF32>(v, w_r, Mul());
        if (p.bias) apply_vec<kVF32>(v, b_r, Add());
        if (p.scale) apply_vec<kVF32>(v, s_r, MulOnePlus());
        if (p.shift) apply_vec<kVF32>(v, t_r, Add());
    } else {
        if (p.weight) apply_vec<kVF32>(v, p.weight, 0, at, Mul());
        if (p.bias) apply_vec<kVF32>(v, p.bias, 0, at, Add());
        if (p.scale) apply_vec<kVF32>(v, p.scale, gbase, at, MulOnePlus());
        if (p.shift) apply_vec<kVF32>(v, p.shift, gbase, at, Add());
    }

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (r < rows) emit<kQuant>(p, row0 + r, base[r], c0 + j * step, at[j], live[j][0], live[j][1], v[r][j]);
        }
}

template <bool kF32, bool kVF32, bool kQuant, int C, int R, bool kFull, bool kEarly>
cudaError_t launch_one(NormParams p, int warps, cudaStream_t stream)
{
    const int64_t groups = ceil_div(p.rows, p.rows_per_group);
    p.row_blocks = groups * ceil_div(p.rows_per_group, R);
    const int64_t grid = p.row_blocks + (kQuant ? p.rows_pad - p.rows : 0);
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    norm_residual_kernel<kF32, kVF32, kQuant, C, R, kFull, kEarly><<<static_cast<unsigned>(grid), 32 * warps, 0, stream>>>(p);
    return cudaGetLastError();
}

// Few rows (two a multiprocessor of the B200's 148): a CTA each, as many warps as a row has spans
// (two spans a warp from 17 on), for the shortest chain of loads.  Many rows: CTAs of at most ten
// warps (more wait longer at each barrier) with one chunk a thread of four rows or, above ten
// spans, two of two rows (of one, for a bf16 stream with bf16 out); rows of more than twenty spans
// take four chunks a thread of one row, and up to 32 warps.
template <bool kF32, bool kVF32, bool kQuant>
cudaError_t launch_shape(const NormParams& p, cudaStream_t stream)
{
    const int spans = static_cast<int>(ceil_div(p.K, 256));
    const bool few = p.rows <= 2 * 148;
    if (few && spans <= 32) {
        if (spans <= 16) return launch_one<kF32, kVF32, kQuant, 1, 1, false, true>(p, spans, stream);
        return launch_one<kF32, kVF32, kQuant, 2, 1, false, true>(p, static_cast<int>(ceil_div(spans, 2)), stream);
    }
    const int c = spans <= 10 ? 1 : spans <= 20 ? 2 : 4;
    const int warps = static_cast<int>(ceil_div(spans, c));
    const bool full = p.K % 256 == 0 && c * warps == spans;
    if (c == 4)
        return full ? launch_one<kF32, kVF32, kQuant, 4, 1, true, false>(p, warps, stream)
                    : launch_one<kF32, kVF32, kQuant, 4, 1, false, false>(p, warps, stream);
    if (c == 1)
        return full ? launch_one<kF32, kVF32, kQuant, 1, 4, true, false>(p, warps, stream)
                    : launch_one<kF32, kVF32, kQuant, 1, 4, false, false>(p, warps, stream);
    constexpr int R = kF32 || kQuant ? 2 : 1;
    return full ? launch_one<kF32, kVF32, kQuant, 2, R, true, false>(p, warps, stream)
                : launch_one<kF32, kVF32, kQuant, 2, R, false, false>(p, warps, stream);
}

}  // namespace

cudaError_t launch_norm_residual(const mxq_norm_desc& d, void* z, int out_fmt, void* out, void* sf,
                                 cudaStream_t stream)
{
    NormParams p = {};
    p.x = d.x;
    p.y = d.y_bf16;
    p.gate = d.gate;
    p.scale = d.scale;
    p.shift = d.shift;
    p.weight = d.weight;
    p.bias = d.bias;
    p.post_weight = d.post_weight;
    p.post_bias = d.post_bias;
    p.z = z;
    p.out = out;
    p.sf = static_cast<uint8_t*>(sf);
    p.rows = d.rows;
    p.K = static_cast<uint32_t>(d.K);
    p.rows_per_group = static_cast<uint32_t>(std::min<int64_t>(d.rows_per_group, d.rows));
    p.atoms_k = static_cast<uint32_t>(sf_atoms_k(d.K));
    p.eps = d.eps;
    p.inv_k = static_cast<float>(1.0 / static_cast<double>(d.K));
    p.norm = d.norm;
    p.post = d.post_norm;
    p.rows_pad = ceil_div(d.rows, 128) * 128;
    p.e4m3 = out_fmt == MXQ_FMT_E4M3;
    const bool f = d.x_dtype == MXQ_DTYPE_F32, vf = d.vec_dtype == MXQ_DTYPE_F32;
    if (out_fmt == MXQ_OUT_BF16) {
        if (f) return vf ? launch_shape<true, true, false>(p, stream) : launch_shape<true, false, false>(p, stream);
        return vf ? launch_shape<false, true, false>(p, stream) : launch_shape<false, false, false>(p, stream);
    }
    if (f) return vf ? launch_shape<true, true, true>(p, stream) : launch_shape<true, false, true>(p, stream);
    return vf ? launch_shape<false, true, true>(p, stream) : launch_shape<false, false, true>(p, stream);
}

}  // namespace mxq
