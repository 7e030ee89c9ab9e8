// gemm_rows.cu -- the residual and gated GEMMs for a few activation rows (up to 64): one
// token, or a batch of decoding sequences.
//
// With few rows the weight is all there is to read (0.53 bytes per element), so the MMA's
// 128-row operand is the weight and its N dimension the tokens: D[n, t] = sum_k W[n, k] x[t, k].
// A 128-row weight tile and one range of K belong to a CTA; the S CTAs of a cluster split K
// and add their partial sums through distributed shared memory, so that every SM streams
// weights even when there are few tiles.  Two CTAs fit an SM.
//   warp 0      TMA producer: weight tile(s), activation rows and their scale atoms into the
//               shared-memory ring;
//   warp 1      allocates TMEM; copies each stage's scales into it (tcgen05.cp) and issues the
//               stage's MMAs (both from one thread, in order);
//   warps 4-7   read the accumulators (lane = weight row, column = token) into shared memory;
// then all warps finish the cluster's tokens, rank r those with t % S == r: sums the S
// partials in rank order (the result does not depend on timing), and applies bias, activation,
// gate and residual, or the gated product and the MX quantization (32 lanes = 32 consecutive
// outputs = one MX block).
// Every wait is bounded; one that runs out records MXQ_ERR_TIMEOUT, the copies in flight are
// waited for, TMEM is freed and no output is written.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdio>

#include "mx_elem.cuh"
#include "mxq_internal.h"
#include "ptx.cuh"

namespace mxq {

__device__ uint32_t g_rows_status;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSplit = 8;  // portable cluster size
constexpr uint64_t kWaitNs = 1000000000ull;

// Operand kinds: W4A4 (kind::mxf4), W4A8 (kind::mxf8f6f4, the weight expanded by TMA to a byte
// an element), bf16 (kind::f16).
constexpr int kMxf4 = 0;
constexpr int kMxf8 = 1;
constexpr int kBf16 = 2;

template <int kKind, bool kGated, int kNT>
struct Cfg {
    static constexpr int kW = kGated ? 2 : 1;                                    // weight tiles a stage
    static constexpr int kAtoms = kKind == kMxf4 ? 2 : kKind == kMxf8 ? 1 : 0;   // scale atoms a stage and operand
    static constexpr int kKps = kKind == kMxf4 ? 256 : kKind == kMxf8 ? 128 : 64;  // K elements a stage
    static constexpr uint32_t kTileW = 128 * 128;
    static constexpr uint32_t kTileX = kNT * 128;
    static constexpr uint32_t kSf = kAtoms * 512;
    static constexpr uint32_t kStage = kW * kTileW + kTileX;
    // As many stages as let two CTAs share an SM's 228 KB (1 KB of each is the system's)
    static constexpr uint32_t kBudget = 115712 - 512;
    static constexpr int kStages = static_cast<int>(kBudget / (kStage + (kW + 1) * kSf));
    static constexpr uint32_t kOffX = kW * kTileW;  // inside a stage
    static constexpr uint32_t kOffSf = kStages * kStage;
    static constexpr uint32_t kOffBar = kOffSf + kStages * (kW + 1) * kSf;
    static constexpr uint32_t kSmem = kOffBar + (2 * kStages + 1) * 8 + 16;
    // bytes a stage's copies report: TMA counts what it writes, except that the expanded
    // weight counts its packed bytes
    static constexpr uint32_t kTx = kW * (kKind == kMxf8 ? kTileW / 2 : kTileW) + kTileX + (kW + 1) * kSf;
    // TMEM: kW accumulators of kNT columns, then 4 columns per scale atom
    static constexpr uint32_t kSfCol = kW * kNT;
    static constexpr uint32_t kCols = kSfCol + (kW + 1) * kAtoms * 4;
    static constexpr uint32_t kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
    static constexpr uint32_t kPart = kW * kNT * 128 * 4;  // fp32 partials, over the stages
    static_assert(kStages >= 2 && kCols <= 256 && kPart <= kStages * kStage, "few-row GEMM plan");
    static_assert(kStage % 1024 == 0, "swizzled tiles are 1024-byte aligned");
    static_assert(3 * (kSmem + 1024) > 233472, "at most two CTAs an SM: they may take half its TMEM each");
};

struct RowsParams {
    int M, N, K, k_stages;
    int act;
    int out_fmt;  // MXQ_OUT_BF16, or the MX format of a gated h
    int gate_f32;
    uint32_t rows_per_group;
    uint32_t atoms_n;  // scale atoms of a quantized h's row
    uint32_t debug;
    const __nv_bfloat16* bias;
    const __nv_bfloat16* bias2;
    const __nv_bfloat16* res;
    const void* gate;
    __nv_bfloat16* y;
    uint8_t* q_codes;
    uint8_t* q_sf;
};

__device__ __forceinline__ void record_status(uint32_t code) { atomicCAS(&g_rows_status, 0u, code); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int kKind, bool kGated, int kNT>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w2,
                     const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_sfw,
                     const __grid_constant__ CUtensorMap map_sfw2, const __grid_constant__ CUtensorMap map_sfx,
                     const RowsParams p)
{
    using C = Cfg<kKind, kGated, kNT>;
    constexpr int S = C::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {  // the same in every CTA
        if (threadIdx.x == 0) record_status(MXQ_ERR_UNSUPPORTED);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* empty = full + S;
    uint64_t* acc_full = full + 2 * S;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(full + 2 * S + 1);
    uint32_t* failed = tmem_base_smem + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = gridDim.x;  // the cluster: one CTA per range of K
    const int rank = blockIdx.x;
    const int tile = blockIdx.y;
    const int ks0 = static_cast<int>(static_cast<int64_t>(p.k_stages) * rank / split);
    const int ks1 = static_cast<int>(static_cast<int64_t>(p.k_stages) * (rank + 1) / split);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<1>(tmem_base_smem, C::kTmem);
        tmem_relinquish<1>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_smem;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            int it = 0;
            bool ok = true;
            int64_t skipped = -1;
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                const int s = it % S;
                if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, kWaitNs)) {
                    ok = false;
                    break;
                }
                if ((p.debug & 1u) && it == 0 && rank == 0 && tile == 0) {
                    skipped = 0;  // deliberately leave the stage unfilled: the MMA wait runs out
                    continue;
                }
                uint8_t* st = smem + s * C::kStage;
                uint8_t* sf = smem + C::kOffSf + s * (C::kW + 1) * C::kSf;
                const uint32_t bar = smem_u32(&full[s]);
                const int kx = kKind == kBf16 ? ks * 64 : ks * 128;  // map elements (bytes, nibbles or bf16)
                mbar_arrive_expect_tx(&full[s], C::kTx);
                tma_load_2d<1>(st, &map_w, kx, tile * 128, bar, pol);
                if constexpr (kGated) tma_load_2d<1>(st + C::kTileW, &map_w2, kx, tile * 128, bar, pol);
                tma_load_2d<1>(st + C::kOffX, &map_x, kx, 0, bar, pol);
                if constexpr (kKind != kBf16) {
                    const int ka = ks * C::kAtoms * 128;  // 32-bit words of the scale rows
                    tma_load_2d<1>(sf, &map_sfw, ka, tile, bar, pol);
                    if constexpr (kGated) tma_load_2d<1>(sf + C::kSf, &map_sfw2, ka, tile, bar, pol);
                    tma_load_2d<1>(sf + C::kW * C::kSf, &map_sfx, ka, 0, bar, pol);
                }
            }
            // every copy issued has landed before this CTA may leave or reuse its memory
            for (int i = max(0, it - S); i < it; ++i)
                if (i != skipped && !mbar_wait(&full[i % S], (i / S) & 1, kWaitNs)) ok = false;
            if (!ok) {
                record_status(MXQ_ERR_TIMEOUT);
                *failed = 1u;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t fw = kKind == kMxf8 ? 5u : 1u;  // weight: E2M1 in both kinds
            constexpr uint32_t fx = kKind == kMxf8 ? 0u : 1u;  // activation: E4M3 / E2M1
            constexpr int kKpm = C::kKps / 4;                  // K elements an MMA
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!mbar_wait(&full[s], ph, kWaitNs)) {
                    record_status(MXQ_ERR_TIMEOUT);
                    *failed = 1u;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * C::kStage);
                const uint32_t sf = smem_u32(smem + C::kOffSf + s * (C::kW + 1) * C::kSf);
                const uint32_t w_lo = sdesc_sw128_lo(st), x_lo = sdesc_sw128_lo(st + C::kOffX);
                const uint32_t tsf = tmem + C::kSfCol;
#pragma unroll
                for (int a = 0; a < (C::kW + 1) * C::kAtoms; ++a)
                    tc_copy_sf_atom<1>(tsf + 4 * a, sdesc_sf_atom(sf + a * 512));
                const int kvalid = p.K - ks * C::kKps;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t accum = ks > ks0 || j > 0 ? 1u : 0u;
#pragma unroll
                    for (int w = 0; w < C::kW; ++w) {
                        const uint32_t wd = w_lo + w * (C::kTileW >> 4) + 2 * j;
                        if constexpr (kKind == kBf16) {
                            mma_bf16<1>(tmem + w * kNT, wd, x_lo + 2 * j, kSdescSw128Hi, idesc_bf16(128, kNT), accum);
                        } else {
                            const uint32_t id = kKind == kMxf8 ? static_cast<uint32_t>(j) : static_cast<uint32_t>((j & 1) * 2);
                            const uint32_t atom = kKind == kMxf8 ? 0u : static_cast<uint32_t>(j >> 1);
                            if (j * kKpm < kvalid)
                                mma_block_scaled<1, kKind == kMxf8>(
                                    tmem + w * kNT, wd, x_lo + 2 * j, kSdescSw128Hi,
                                    idesc_block_scaled(fw, fx, 128, kNT, id, id), tsf + 4 * (w * C::kAtoms + atom),
                                    tsf + 4 * (C::kW * C::kAtoms + atom), accum);
                        }
                    }
                }
                tc_commit<1>(&empty[s]);
                if (++s == S) { s = 0; ph ^= 1; }
            }
            tc_commit<1>(acc_full);  // also after a time-out: whatever was issued completes first
            if (!mbar_wait(acc_full, 0, kWaitNs) && ok) {
                record_status(MXQ_ERR_TIMEOUT);
                *failed = 1u;
            }
        }
    }
    // all MMAs are done and all copies landed; the stages' memory now holds the partials
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    float* part = reinterpret_cast<float*>(smem);  // [kW][kNT][128]
    if (warp >= 4) {
        const int q = warp & 3;  // TMEM lane quarter this warp may access
#pragma unroll
        for (int w = 0; w < C::kW; ++w)
#pragma unroll 1
            for (int t0 = 0; t0 < kNT; t0 += 16) {
                if (t0 >= p.M) break;
                uint32_t r[16];
                tmem_ld_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + w * kNT + t0, r);
                tmem_ld_wait();
                tmem_regs_ready(r);
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t0 + t < p.M) part[(w * kNT + t0 + t) * 128 + q * 32 + lane] = __uint_as_float(r[t]);
            }
        tc_fence_before();
    }
    cluster_sync();  // the cluster's partials are written (and TMEM is read)
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(tmem, C::kTmem);

    bool ok = true;
    const uint32_t flag = smem_u32(failed);
    const uint32_t mine = smem_u32(part);
    for (int r = 0; r < split; ++r) {
        const float f = ld_cluster_f32(mapa_shared(flag, r));
        ok = ok && __float_as_uint(f) == 0u;
    }
    if (ok) {
        const int nq = tile * 128 + (warp & 3) * 32;  // this warp's 32 output columns
        const int n = nq + lane;
        const bool live = n < p.N;
        const float b0 = p.bias != nullptr && live ? __bfloat162float(p.bias[n]) : 0.0f;
        const float b1 = kGated && p.bias2 != nullptr && live ? __bfloat162float(p.bias2[n]) : 0.0f;
        with_act(p.act, [&](auto act) {
            for (int t = rank + split * (warp >> 2); t < p.M; t += split * 2) {
                float v[C::kW];
#pragma unroll
                for (int w = 0; w < C::kW; ++w) {
                    const uint32_t off = ((w * kNT + t) * 128 + (warp & 3) * 32 + lane) * 4;
                    float a[kMaxSplit];
#pragma unroll
                    for (int r = 0; r < kMaxSplit; ++r)
                        a[r] = r < split ? ld_cluster_f32(mapa_shared(mine + off, r)) : 0.0f;
                    v[w] = a[0];
#pragma unroll
                    for (int r = 1; r < kMaxSplit; ++r) v[w] += a[r];
                }
                float o = act_f32<act>(v[0] + b0);
                if constexpr (kGated) {
                    o *= v[C::kW - 1] + b1;
                } else {
                    if (p.gate != nullptr && live) {
                        const size_t gi = static_cast<size_t>(static_cast<uint32_t>(t) / p.rows_per_group) * p.N + n;
                        o *= p.gate_f32 ? static_cast<const float*>(p.gate)[gi]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.gate)[gi]);
                    }
                    if (p.res != nullptr && live) o += __bfloat162float(p.res[static_cast<size_t>(t) * p.N + n]);
                }
                if (!kGated || p.out_fmt == MXQ_OUT_BF16) {
                    if (live) p.y[static_cast<size_t>(t) * p.N + n] = __float2bfloat16_rn(o);
                    continue;
                }
                // h: the warp's 32 values of this token are one MX block (N is a multiple of 32)
                uint32_t sc = 0u;
                if (nq < p.N) {
                    const uint32_t hb = bf16x2_bits(o, o);
                    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, hb & 0x7FFFu);
                    const bool e4m3 = p.out_fmt == MXQ_FMT_E4M3;
                    sc = e4m3 ? e8m0_code<8u>(m) : e8m0_code<2u>(m);
                    const float q = lo_f(hb) * e8m0_inverse(sc);
                    const float q1 = __shfl_down_sync(0xFFFFFFFFu, q, 1);
                    if (e4m3) {
                        p.q_codes[static_cast<size_t>(t) * p.N + n] =
                            sc == 255u ? uint8_t(0) : static_cast<uint8_t>(cvt_e4m3x2(q, 0.0f) & 0xFFu);
                    } else if ((lane & 1) == 0) {
                        const float pair[8] = {q, q1, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        p.q_codes[(static_cast<size_t>(t) * p.N + n) / 2] =
                            sc == 255u ? uint8_t(0) : static_cast<uint8_t>(cvt_e2m1x8(pair) & 0xFFu);
                    }
                }
                if (lane == 0)  // this token's scale byte (0 for the padding past N)
                    p.q_sf[sf_word(t, tile, p.atoms_n) + (warp & 3)] = static_cast<uint8_t>(sc);
            }
        });
        if (kGated && p.out_fmt != MXQ_OUT_BF16)  // the layout's padding rows, one word of this tile each
            for (int t = p.M + rank * kThreads + static_cast<int>(threadIdx.x); t < 128; t += split * kThreads)
                *reinterpret_cast<uint32_t*>(p.q_sf + sf_word(t, tile, p.atoms_n)) = 0u;
    }
    cluster_sync();  // no CTA leaves while another may read its partials
}

template <int kKind, bool kGated, int kNT>
cudaError_t launch_rows(const CUtensorMap (&m)[6], const RowsParams& p, int split, int tiles, cudaStream_t stream)
{
    using C = Cfg<kKind, kGated, kNT>;
    auto kern = gemm_rows_kernel<kKind, kGated, kNT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split, tiles, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], m[3], m[4], m[5], p);
}

template <int kKind, bool kGated>
cudaError_t launch_nt(int nt, const CUtensorMap (&m)[6], const RowsParams& p, int split, int tiles,
                      cudaStream_t stream)
{
    if (nt == 16) return launch_rows<kKind, kGated, 16>(m, p, split, tiles, stream);
    if (nt == 32) return launch_rows<kKind, kGated, 32>(m, p, split, tiles, stream);
    return launch_rows<kKind, kGated, 64>(m, p, split, tiles, stream);
}

template <int kKind>
cudaError_t launch_kind(bool gated, int nt, const CUtensorMap (&m)[6], const RowsParams& p, int split, int tiles,
                        cudaStream_t stream)
{
    return gated ? launch_nt<kKind, true>(nt, m, p, split, tiles, stream)
                 : launch_nt<kKind, false>(nt, m, p, split, tiles, stream);
}

}  // namespace

int read_and_clear_rows_status(cudaStream_t stream, uint32_t* out)
{
    uint32_t v = 0, zero = 0;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return MXQ_ERR_CUDA;
    if (cudaMemcpyFromSymbol(&v, g_rows_status, sizeof v) != cudaSuccess) return MXQ_ERR_CUDA;
    if (cudaMemcpyToSymbol(g_rows_status, &zero, sizeof zero) != cudaSuccess) return MXQ_ERR_CUDA;
    *out = v;
    return MXQ_OK;
}

int launch_gemm_rows(const GemmArgs& g, cudaStream_t stream, const char** msg, char* path, size_t path_len)
{
    const bool gated = g.epilogue == kEpilogueGated;
    const int kind = g.bf16 ? kBf16 : g.a_fmt == kFmtE4M3 ? kMxf8 : kMxf4;
    const int nt = g.M <= 16 ? 16 : g.M <= 32 ? 32 : 64;
    const int64_t atoms_k = sf_atoms_k(g.K);
    const uint32_t ak = kind == kMxf4 ? 2 : 1;
    CUtensorMap m[6];
    bool ok = true;
    auto weight = [&](CUtensorMap* t, const void* w) {
        if (kind == kBf16)
            return make_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w, g.K, g.N, g.K * 2, 64, 128,
                               CU_TENSOR_MAP_SWIZZLE_128B);
        if (kind == kMxf8)
            return make_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, w, g.K, g.N, g.K / 2, 128, 128,
                               CU_TENSOR_MAP_SWIZZLE_128B);
        return make_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, g.K / 2, g.N, g.K / 2, 128, 128,
                           CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto scales = [&](CUtensorMap* t, const void* sf, int64_t rows) {
        return make_map_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT32, sf, atoms_k * 128, ceil_div(rows, 128), atoms_k * 512,
                           ak * 128, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    ok = weight(&m[0], g.w_codes);
    if (gated) ok = ok && weight(&m[1], g.w2_codes);
    else m[1] = m[0];
    if (kind == kBf16) {
        ok = ok && make_map_2d(&m[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.a_codes, g.K, g.M, g.K * 2, 64, nt,
                               CU_TENSOR_MAP_SWIZZLE_128B);
        m[3] = m[4] = m[5] = m[0];  // never used
    } else {
        const uint64_t row = kind == kMxf8 ? g.K : g.K / 2;
        ok = ok && make_map_2d(&m[2], CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a_codes, row, g.M, row, 128, nt,
                               CU_TENSOR_MAP_SWIZZLE_128B);
        ok = ok && scales(&m[3], g.w_sf, g.N);
        if (gated) ok = ok && scales(&m[4], g.w2_sf, g.N);
        else m[4] = m[3];
        ok = ok && scales(&m[5], g.a_sf, g.M);
    }
    if (!ok) {
        *msg = "cuTensorMapEncodeTiled failed (driver entry point unavailable or invalid operand layout)";
        return MXQ_ERR_CUDA;
    }
    RowsParams p = {};
    p.M = static_cast<int>(g.M);
    p.N = static_cast<int>(g.N);
    p.K = static_cast<int>(g.K);
    p.k_stages = static_cast<int>(ceil_div(g.K, kind == kMxf4 ? 256 : kind == kMxf8 ? 128 : 64));
    p.act = g.act;
    p.out_fmt = g.out_fmt;
    p.gate_f32 = g.gate_f32 ? 1 : 0;
    p.rows_per_group = static_cast<uint32_t>(std::min<int64_t>(g.rows_per_group, g.M));
    p.atoms_n = static_cast<uint32_t>(sf_atoms_k(g.N));
    p.debug = debug_flags();
    p.bias = static_cast<const __nv_bfloat16*>(g.bias);
    p.bias2 = static_cast<const __nv_bfloat16*>(g.bias2);
    p.res = static_cast<const __nv_bfloat16*>(g.residual);
    p.gate = g.gate;
    p.y = static_cast<__nv_bfloat16*>(g.y);
    p.q_codes = static_cast<uint8_t*>(g.q_codes);
    p.q_sf = static_cast<uint8_t*>(g.q_sf);

    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // K is split while all CTAs still run at once, two to an SM
    const int tiles = static_cast<int>(ceil_div(g.N, 128));
    int split = 1;
    while (split < kMaxSplit && 2 * split * tiles <= 2 * sms && 2 * split <= p.k_stages) split *= 2;
    cudaError_t e = kind == kBf16   ? launch_kind<kBf16>(gated, nt, m, p, split, tiles, stream)
                    : kind == kMxf8 ? launch_kind<kMxf8>(gated, nt, m, p, split, tiles, stream)
                                    : launch_kind<kMxf4>(gated, nt, m, p, split, tiles, stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        *msg = cudaGetErrorString(e);
        return MXQ_ERR_CUDA;
    }
    if (path)
        snprintf(path, path_len, "rows %s 128x%d split %d tiles %d%s", kind == kBf16 ? "bf16" : kind == kMxf8 ? "mxf8f6f4" : "mxf4",
                 nt, split, tiles, epilogue_name(g));
    return MXQ_OK;
}

}  // namespace mxq
