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
// row in registers (first the mean, then the centered squares), so a large common offset
// costs no digits.
//
// One CTA per row, the row in registers (C chunks of 8 channels a thread): x and y are read
// once and z and h written once, which is all the traffic there is; HBM bounds it.  The
// per-channel vectors (gate, scale, shift, weights) are shared by all rows of a group and
// come from L1.
#include <cuda_bf16.h>

#include <algorithm>

#include "mx_elem.cuh"
#include "mxq_internal.h"

namespace mxq {

namespace {

constexpr int kMaxThreads = 512;

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
    uint32_t K;
    uint32_t rows_per_group;
    uint32_t atoms_k;
    float eps;
    float inv_k;
    int norm, post;  // MXQ_NORM_*
    int vec_f32;     // the per-channel vectors are fp32 (else bf16)
};

// Eight consecutive channels of a bf16 or fp32 array, as they lie in memory.
struct Raw8 {
    uint4 a, b;
};

__device__ __forceinline__ Raw8 load_vec8(const void* p, size_t i, bool f32)
{
    Raw8 r;
    if (f32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        r.a = __ldg(q);
        r.b = __ldg(q + 1);
    } else {
        r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
        r.b = make_uint4(0u, 0u, 0u, 0u);
    }
    return r;
}

__device__ __forceinline__ void widen8(const Raw8& r, bool f32, float (&v)[8])
{
    if (f32) {
        v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
        v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
        v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
        v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
    } else {
        v[0] = lo_f(r.a.x); v[1] = hi_f(r.a.x);
        v[2] = lo_f(r.a.y); v[3] = hi_f(r.a.y);
        v[4] = lo_f(r.a.z); v[5] = hi_f(r.a.z);
        v[6] = lo_f(r.a.w); v[7] = hi_f(r.a.w);
    }
}

// The rows themselves are read once: streaming loads, which leave L1 to the vectors.
template <bool kF32>
__device__ __forceinline__ Raw8 load_row8(const void* p, size_t i)
{
    Raw8 r;
    if (kF32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        r.a = __ldcs(q);
        r.b = __ldcs(q + 1);
    } else {
        r.a = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
        r.b = make_uint4(0u, 0u, 0u, 0u);
    }
    return r;
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
}

// Sum over the CTA, the same value in every thread.  `red` is used by this call only.
__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);  // at most 16 warps
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// Mean (0 for RMSNorm) and 1 / sqrt(variance + eps) of the CTA's row, whose channels past K
// are held as zeros and masked out of the centered squares by `live`.
template <int C>
__device__ __forceinline__ float2 row_stats(const float (&v)[C][8], const bool (&live)[C], int kind, float inv_k,
                                            float eps, float* red)
{
    float mean = 0.0f;
    if (kind == MXQ_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[j][i];
        mean = block_sum(s, red) * inv_k;
    }
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        if (!live[j]) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = v[j][i] - mean;
            q = fmaf(d, d, q);
        }
    }
    const float var = block_sum(q, red + 16) * inv_k;
    return make_float2(mean, __frsqrt_rn(var + eps));
}

// kF32: the residual stream x, z is fp32 (else bf16).  OUT: MXQ_OUT_BF16, MXQ_FMT_E2M1 or
// MXQ_FMT_E4M3.  C: chunks of 8 channels per thread; chunk j of thread t is chunk j * T + t of
// the row, so four neighbouring lanes hold one MX block.
template <bool kF32, int OUT, int C>
__global__ void __launch_bounds__(kMaxThreads) norm_residual_kernel(const NormParams p)
{
    __shared__ float red[64];
    const int64_t row = blockIdx.x;
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t chunks = p.K / 8;
    const bool vf = p.vec_f32 != 0;
    if constexpr (OUT != MXQ_OUT_BF16) {
        if (row >= p.rows) {  // a row of the scale layout's padding
            for (uint32_t a = threadIdx.x; a < p.atoms_k; a += blockDim.x)
                *reinterpret_cast<uint32_t*>(p.sf + sf_word(row, a, p.atoms_k)) = 0u;
            return;
        }
    }
    const size_t base = static_cast<size_t>(row) * p.K;
    const size_t gbase = static_cast<size_t>(static_cast<uint32_t>(row) / p.rows_per_group) * p.K;

    bool live[C];
    uint32_t ch[C];  // first channel of each chunk
    Raw8 xr[C], yr[C];
    float v[C][8];   // the row: y (with a post norm), then z
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const uint32_t c = j * blockDim.x + threadIdx.x;
        live[j] = c < chunks;
        ch[j] = c * 8u;
        xr[j].a = xr[j].b = yr[j].a = yr[j].b = make_uint4(0u, 0u, 0u, 0u);
        if (live[j]) {
            xr[j] = load_row8<kF32>(p.x, base + ch[j]);
            if (p.y) yr[j] = load_row8<false>(p.y, base + ch[j]);
        }
    }
    // up to two chunks a thread: the vectors of the last step are fetched here too, so that
    // their latency passes beside the row's (a call of few rows is bound by nothing else)
    constexpr bool kEarly = C <= 2;
    Raw8 w_r[kEarly ? C : 1], b_r[kEarly ? C : 1], s_r[kEarly ? C : 1], t_r[kEarly ? C : 1];
    if constexpr (kEarly) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (!live[j]) continue;
            if (p.weight) w_r[j] = load_vec8(p.weight, ch[j], vf);
            if (p.bias) b_r[j] = load_vec8(p.bias, ch[j], vf);
            if (p.scale) s_r[j] = load_vec8(p.scale, gbase + ch[j], vf);
            if (p.shift) t_r[j] = load_vec8(p.shift, gbase + ch[j], vf);
        }
    }

    if (p.y) {
        float2 st = make_float2(0.0f, 1.0f);
        if (p.post != MXQ_NORM_NONE) {
#pragma unroll
            for (int j = 0; j < C; ++j) widen8(yr[j], false, v[j]);
            st = row_stats<C>(v, live, p.post, p.inv_k, p.eps, red + 32);
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float xv[8], t[8];
            widen8(xr[j], kF32, xv);
            widen8(yr[j], false, v[j]);
            if (live[j]) {
                if (p.post != MXQ_NORM_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] - st.x) * st.y;
                    if (p.post_weight) {
                        widen8(load_vec8(p.post_weight, ch[j], vf), vf, t);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] *= t[i];
                    }
                    if (p.post_bias) {
                        widen8(load_vec8(p.post_bias, ch[j], vf), vf, t);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[j][i] += t[i];
                    }
                }
                if (p.gate) {
                    widen8(load_vec8(p.gate, gbase + ch[j], vf), vf, t);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = fmaf(t[i], v[j][i], xv[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] += xv[i];
                }
                if constexpr (kF32) {
                    float4* zp = reinterpret_cast<float4*>(static_cast<float*>(p.z) + base + ch[j]);
                    zp[0] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
                    zp[1] = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
                } else {
                    Raw8 zr;
                    zr.a = pack8(v[j]);
                    zr.b = zr.a;
                    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.z) + base + ch[j]) = zr.a;
                    widen8(zr, false, v[j]);  // the norm sees the stored value
                }
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) widen8(xr[j], kF32, v[j]);
    }

    const float2 st = row_stats<C>(v, live, p.norm, p.inv_k, p.eps, red);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = (v[j][i] - st.x) * st.y;
        if (live[j]) {
            if (p.weight) {
                widen8(kEarly ? w_r[kEarly ? j : 0] : load_vec8(p.weight, ch[j], vf), vf, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] *= t[i];
            }
            if (p.bias) {
                widen8(kEarly ? b_r[kEarly ? j : 0] : load_vec8(p.bias, ch[j], vf), vf, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += t[i];
            }
            if (p.scale) {
                widen8(kEarly ? s_r[kEarly ? j : 0] : load_vec8(p.scale, gbase + ch[j], vf), vf, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * (1.0f + t[i]);
            }
            if (p.shift) {
                widen8(kEarly ? t_r[kEarly ? j : 0] : load_vec8(p.shift, gbase + ch[j], vf), vf, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] += t[i];
            }
        }
        const uint4 o = pack8(v[j]);
        if constexpr (OUT == MXQ_OUT_BF16) {
            if (live[j]) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + base + ch[j]) = o;
        } else {
            // the quad's 32 values are one MX block: the activation quantizer's arithmetic on
            // the bf16 h (scale from the abs-max's exponent field, codes rounded to nearest
            // even with saturation, zero codes in a non-finite block)
            constexpr uint32_t kEmax = OUT == MXQ_FMT_E4M3 ? 8u : 2u;
            uint32_t m = absmax_bf16x2(absmax_bf16x2(o.x, o.y), absmax_bf16x2(o.z, o.w));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            m = absmax_bf16x2(m, __byte_perm(m, 0, 0x1032));
            const uint32_t sc = e8m0_code<kEmax>(m);
            const float inv = e8m0_inverse(sc);
            const uint32_t keep = sc == 255u ? 0u : 0xFFFFFFFFu;
            // four blocks' scale bytes (16 lanes) make one word of the tiled layout
            const uint32_t kb = ch[j] / 32u;
            uint32_t word = live[j] ? sc << (8u * (kb & 3u)) : 0u;
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
            word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
            float q[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = i == 0 ? o.x : i == 1 ? o.y : i == 2 ? o.z : o.w;
                q[2 * i] = lo_f(w) * inv;
                q[2 * i + 1] = hi_f(w) * inv;
            }
            if (live[j]) {
                uint8_t* codes = static_cast<uint8_t*>(p.out);
                if constexpr (OUT == MXQ_FMT_E2M1) {
                    *reinterpret_cast<uint32_t*>(codes + (base + ch[j]) / 2) = cvt_e2m1x8(q) & keep;
                } else {
                    const uint32_t c0 = (cvt_e4m3x2(q[0], q[1]) | (cvt_e4m3x2(q[2], q[3]) << 16)) & keep;
                    const uint32_t c1 = (cvt_e4m3x2(q[4], q[5]) | (cvt_e4m3x2(q[6], q[7]) << 16)) & keep;
                    *reinterpret_cast<uint2*>(codes + base + ch[j]) = make_uint2(c0, c1);
                }
                // k-blocks past K inside the word stay 0, as the layout's padding requires
                if ((lane & 15u) == 0) *reinterpret_cast<uint32_t*>(p.sf + sf_word(row, kb / 4u, p.atoms_k)) = word;
            }
        }
    }
}

template <bool kF32, int OUT>
cudaError_t launch_c(int c, unsigned grid, int threads, const NormParams& p, cudaStream_t stream)
{
    if (c == 1) norm_residual_kernel<kF32, OUT, 1><<<grid, threads, 0, stream>>>(p);
    else if (c == 2) norm_residual_kernel<kF32, OUT, 2><<<grid, threads, 0, stream>>>(p);
    else if (c <= 4) norm_residual_kernel<kF32, OUT, 4><<<grid, threads, 0, stream>>>(p);
    else norm_residual_kernel<kF32, OUT, 8><<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <bool kF32>
cudaError_t launch_out(int out, int c, unsigned grid, int threads, const NormParams& p, cudaStream_t stream)
{
    if (out == MXQ_FMT_E2M1) return launch_c<kF32, MXQ_FMT_E2M1>(c, grid, threads, p, stream);
    if (out == MXQ_FMT_E4M3) return launch_c<kF32, MXQ_FMT_E4M3>(c, grid, threads, p, stream);
    return launch_c<kF32, MXQ_OUT_BF16>(c, grid, threads, p, stream);
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
    p.vec_f32 = d.vec_dtype == MXQ_DTYPE_F32;
    // Few rows: as many threads as the row has chunks, for the shortest chain of loads.  Many
    // rows: four chunks a thread, which keeps more bytes in flight per register.
    const int chunks = p.K / 8;
    const bool few = d.rows <= 2 * 148;
    const int want = few ? chunks : std::max(64, static_cast<int>(ceil_div(chunks, 4)));
    const int threads = std::min<int>(kMaxThreads, static_cast<int>(ceil_div(want, 32)) * 32);
    const int c = static_cast<int>(ceil_div(chunks, threads));
    const bool quant = out_fmt != MXQ_OUT_BF16;
    const unsigned grid = static_cast<unsigned>(quant ? ceil_div(d.rows, 128) * 128 : d.rows);
    return d.x_dtype == MXQ_DTYPE_F32 ? launch_out<true>(out_fmt, c, grid, threads, p, stream)
                                      : launch_out<false>(out_fmt, c, grid, threads, p, stream);
}

}  // namespace mxq
