// gemm_rows.cu -- the residual and gated GEMMs for few activation rows: one token, a batch of
// decoding sequences, a short prompt (few_rows in mxq_internal.h draws the line).
//
// With few rows the weight is all there is to read (0.53 bytes per element), so the MMA's
// 128-row operand is the weight and its N dimension the tokens: D[n, t] = sum_k W[n, k] x[t, k].
// A 128-row weight tile, up to 64 tokens and one range of K belong to a CTA; the S CTAs of a cluster split K
// and add their partial sums through distributed shared memory, so that every SM streams
// weights even when there are few tiles.  Two CTAs fit an SM.
//   warp 0      TMA producer: weight tile(s), activation rows and their scale atoms into the
//               shared-memory ring; it fills the ring before the rest of the CTA is set up;
//   warp 1      allocates TMEM and issues each stage's MMAs;
//   warps 2, 3  copy each stage's scales into the stage's own TMEM columns (tcgen05.cp) ahead of
//               the MMAs, the weights' and the activation's;
//   warps 4-7   (kQX: up to 16 rows of bf16 x) quantize each stage's part of x straight into the
//               stage, a launch and a round trip through memory less;
//   warps 4-7   read the accumulators (lane = weight row, column = token) into shared memory;
// then all warps finish the cluster's tokens in fours, rank a % S the a-th four: read the S
// partials (one 16-byte load a rank), add them in rank order (the result does not depend on
// timing), and apply bias, activation, gate and residual, or the gated product and the MX
// quantization (32 lanes = 32 consecutive outputs = one MX block).
// Launches are programmatic: the set-up runs while the kernel before on the stream ends.  All
// global reads and writes come after griddepcontrol.wait (by plain loads: the non-coherent path is for
// data that nothing writes while the kernel runs, and the compiler may move such a load), except that behind a kernel of the same
// call (the quantizer of x, or the gated network's first kernel) the weight is read before it: the
// quantizer is an ordinary launch and the first kernel lets this one start only after its own wait,
// so whatever wrote the weight has completed.  (48 rows of 5120 x 13824 W4A8, quantizer included:
// 19.2 us with K split in 4, 20.3 without.)
// Measured (kernel time in a loop, weights not in L2): one row of 5120 x 5120 W4A4 7.2 us, 48 rows
// 8.9; 48 rows of 5120 x 13824 W4A8 14.5 us; gated, one row of both 13824 x 5120 weights 18.0 us (4.2
// TB/s).  Bound by latency: set-up, the first stage's round trip and the cluster's reduction are 5 us.
// Every wait is bounded; one that runs out records MXQ_ERR_TIMEOUT, the copies in flight are
// waited for, TMEM is freed and no output is written.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
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
    static constexpr uint32_t kPart = kW * kNT * 128 * 4;  // a CTA's partial sums, over its stages
    // As many stages as let two CTAs share an SM's 228 KB (1 KB of each is the system's)
    static constexpr uint32_t kBudget = 115712 - 512;
    static constexpr int kStages = static_cast<int>(kBudget / (kStage + (kW + 1) * kSf));
    static constexpr uint32_t kOffX = kW * kTileW;  // inside a stage
    static constexpr uint32_t kOffSf = kStages * kStage;  // [operand][stage][kSf], the weights first
    static constexpr uint32_t kOffBar = kOffSf + kStages * (kW + 1) * kSf;
    static constexpr uint32_t kSmem = kOffBar + (3 * kStages + 1) * 8 + 16;
    // bytes a stage's tensor copies report: TMA counts what it writes, except that the
    // expanded weight counts its packed bytes
    static constexpr uint32_t kTxW = kW * (kKind == kMxf8 ? kTileW / 2 : kTileW);
    // TMEM: kW accumulators of kNT columns, then each stage's scales, 4 columns an atom
    static constexpr uint32_t kSfCol = kW * kNT;
    static constexpr uint32_t kSfCols = (kW + 1) * kAtoms * 4;
    static constexpr uint32_t kCols = kSfCol + kStages * kSfCols;
    static constexpr uint32_t kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : 256;
    static_assert(kStages >= 2 && kCols <= 256 && kPart <= kStages * kStage, "few-row GEMM plan");
    static_assert(kStage % 1024 == 0, "swizzled tiles are 1024-byte aligned");
    static_assert(3 * (kSmem + 1024) > 233472, "at most two CTAs an SM: they may take half its TMEM each");
};

struct RowsParams {
    int M, N, K, k_stages;
    int split;  // the cluster: one CTA per range of K
    int act;
    int out_fmt;  // MXQ_OUT_BF16, or the MX format of a gated h
    int gate_f32;
    uint32_t rows_per_group;
    uint32_t atoms_n;  // scale atoms of a quantized h's row
    uint32_t debug;
    const uint8_t* sf_w;   // tiled scales: the weight's, the second weight's, the activation's
    const uint8_t* sf_w2;
    const uint8_t* sf_x;
    uint32_t atoms_k;      // scale atoms of a row of K
    int early;         // the weight may be read before the kernel before on the stream has ended
    const __nv_bfloat16* x;  // kQX: the activation, quantized on the way
    const __nv_bfloat16* bias;
    const __nv_bfloat16* bias2;
    const __nv_bfloat16* res;
    const void* gate;
    __nv_bfloat16* y;
    uint8_t* q_codes;
    uint8_t* q_sf;
};

__device__ __forceinline__ void record_status(uint32_t code) { atomicCAS(&g_rows_status, 0u, code); }

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Quantizes rows x[0 .. M) of one stage (kKps columns from k0) into the stage's operand tile
// (128-byte rows under the 128-byte swizzle) and scale atoms, with the activation quantizer's
// arithmetic.  Four lanes take one MX block.  Blocks past K get zero codes and scales (the
// MMA's other operand is zero there, and 0 x NaN must not reach the sum); tile rows past M are
// left as they are, since they only reach output columns that nothing reads.
template <int kKind>
struct QuantX {
    static constexpr int kKps = kKind == kMxf4 ? 256 : 128;
    static constexpr int kLanes = kKps / 8;                // lanes a row
    static constexpr int kRounds = 16 * kLanes / 128;      // of 128 threads, for 16 rows
    uint4 raw[kRounds];

    __device__ __forceinline__ void load(const RowsParams& p, int ks, int tid)
    {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int unit = i * 128 + tid, row = unit / kLanes, k = ks * kKps + unit % kLanes * 8;
            raw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < p.M && k < p.K) raw[i] = *reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(row) * p.K + k);
        }
    }

    __device__ __forceinline__ void store(const RowsParams& p, int ks, int tid, uint8_t* tile, uint8_t* sf) const
    {
        constexpr uint32_t kEmax = kKind == kMxf8 ? 8u : 2u;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int unit = i * 128 + tid, row = unit / kLanes, kl = unit % kLanes * 8;
            if ((i * 128 + (tid & ~31)) / kLanes >= p.M) break;  // warp-uniform: no row of this warp is live
            const uint4 o = raw[i];
            uint32_t m = absmax_bf16x2(absmax_bf16x2(o.x, o.y), absmax_bf16x2(o.z, o.w));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            m = absmax_bf16x2(m, __byte_perm(m, 0, 0x1032));
            const uint32_t sc = e8m0_code<kEmax>(m);
            const float inv = e8m0_inverse(sc);
            const uint32_t keep = sc == 255u ? 0u : 0xFFFFFFFFu;
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
            float q[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                q[2 * j] = lo_f(w[j]) * inv;
                q[2 * j + 1] = hi_f(w[j]) * inv;
            }
            if (row < p.M) {
                const uint32_t byte = static_cast<uint32_t>(kKind == kMxf8 ? kl : kl / 2);
                uint8_t* at = tile + row * 128 + (((byte >> 4) ^ (static_cast<uint32_t>(row) & 7u)) << 4) + (byte & 15u);
                if constexpr (kKind == kMxf8) {
                    const uint32_t c0 = (cvt_e4m3x2(q[0], q[1]) | (cvt_e4m3x2(q[2], q[3]) << 16)) & keep;
                    const uint32_t c1 = (cvt_e4m3x2(q[4], q[5]) | (cvt_e4m3x2(q[6], q[7]) << 16)) & keep;
                    *reinterpret_cast<uint2*>(at) = make_uint2(c0, c1);
                } else {
                    *reinterpret_cast<uint32_t*>(at) = cvt_e2m1x8(q) & keep;
                }
                if ((tid & 3) == 0) sf[(kl / 128) * 512 + row * 16 + (kl / 32 & 3)] = static_cast<uint8_t>(sc);
            }
        }
    }
};

template <int kKind, bool kGated, int kNT, bool kQX>
__global__ void __launch_bounds__(kThreads, 2)
    gemm_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w2,
                     const __grid_constant__ CUtensorMap map_x, const RowsParams p)
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
    uint64_t* sf_ready = full + 2 * S;  // a stage's scales are in TMEM (and so the stage has landed)
    uint64_t* acc_full = full + 3 * S;
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(full + 3 * S + 1);
    uint32_t* failed = tmem_base_smem + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = static_cast<int>(cluster_ctarank());
    const int tile = static_cast<int>(cluster_id_x());
    const int m0 = blockIdx.y * kNT;  // the CTA's tokens
    const int M = min(kNT, p.M - m0);
    const int ks0 = static_cast<int>(static_cast<int64_t>(p.k_stages) * rank / split);
    const int ks1 = static_cast<int>(static_cast<int64_t>(p.k_stages) * (rank + 1) / split);
    const int n_stages = ks1 - ks0;
    const int n_first = min(S, n_stages);  // the ring starts out empty
    // debug: leave one stage unfilled, so that the MMA wait runs out
    const int skipped = (p.debug & 1u) && rank == 0 && tile == 0 && m0 == 0 ? 0 : -1;

    // one operand's scale bytes in the CTA's stage `it` (the last stage of K may have fewer atoms)
    auto sf_bytes_of = [&](int it) {
        const int a0 = (ks0 + it) * C::kAtoms;
        return static_cast<uint32_t>(min(C::kAtoms, static_cast<int>(p.atoms_k) - a0)) * 512u;
    };
    // operand o's scales (0, 1: the weights; kW: the activation) of a stage: one contiguous run
    auto load_sf = [&](int o, int it) {
        const uint8_t* base = o == C::kW ? p.sf_x : o == 0 ? p.sf_w : p.sf_w2;
        const size_t row = static_cast<size_t>(o == C::kW ? m0 / 128 : tile) * p.atoms_k * 512u;
        bulk_load(smem + C::kOffSf + (o * S + it % S) * C::kSf, base + row + static_cast<size_t>(ks0 + it) * C::kSf,
                  sf_bytes_of(it), smem_u32(&full[it % S]));
    };
    constexpr int kSfOps = C::kW + (kQX ? 0 : 1);  // operands whose scales are loaded
    auto expect = [&](int it) {
        mbar_arrive_expect_tx(&full[it % S], C::kTxW + (kQX ? 0u : C::kTileX) +
                                                 (kKind != kBf16 ? kSfOps * sf_bytes_of(it) : 0u));
    };
    auto load_w = [&](int it, uint64_t pol) {
        uint8_t* st = smem + it % S * C::kStage;
        const uint32_t bar = smem_u32(&full[it % S]);
        const int kx = (ks0 + it) * (kKind == kBf16 ? 64 : 128);  // map elements (bytes, nibbles or bf16)
        tma_load_2d<1>(st, &map_w, kx, tile * 128, bar, pol);
        if constexpr (kGated) tma_load_2d<1>(st + C::kTileW, &map_w2, kx, tile * 128, bar, pol);
    };
    auto load_x = [&](int it, uint64_t pol) {
        tma_load_2d<1>(smem + it % S * C::kStage + C::kOffX, &map_x, (ks0 + it) * (kKind == kBf16 ? 64 : 128), m0,
                       smem_u32(&full[it % S]), pol);
    };

    uint64_t pol = 0;
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1 + (kQX ? 4 : 0));  // the copies, and the quantizing warps
        fence_mbar_init();
        pol = policy_evict_normal();
        if (!p.early) grid_wait();
        for (int it = 0; it < n_first; ++it) {
            if (it == skipped) continue;
            expect(it);
            load_w(it, pol);
            if constexpr (kKind != kBf16)
                for (int o = 0; o < C::kW; ++o) load_sf(o, it);
        }
    }
    if (warp == 1) {
        tmem_alloc<1>(tmem_base_smem, C::kTmem);
        tmem_relinquish<1>();
    }
    if (warp == 2 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&empty[s], 1);
            mbar_init(&sf_ready[s], 2);  // the weights' scales, and the activation's
        }
        mbar_init(acc_full, 1);
        *failed = 0u;
        fence_mbar_init();
    }
    if (warp == 3 && lane == 0) {
        prefetch_tmap(&map_w);
        if (kGated) prefetch_tmap(&map_w2);
        if (!kQX) prefetch_tmap(&map_x);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_smem;

    const int nq = tile * 128 + (warp & 3) * 32;  // the 32 output columns this warp finishes
    const int n = nq + lane;
    const bool live = n < p.N;
    // Tokens are finished in fours: four a by rank a % split, its warps 0-3 and 4-7 taking
    // alternate ones of the rank's.  first4: this warp's first four.
    const int first4 = rank + split * (warp >> 2);
    // As loaded, so that nothing waits for the loads before the last step: bf16 bits in the low
    // half, or a gate's fp32 bits.
    uint32_t bias_r[2] = {0u, 0u}, gate_r[4], res_r[4];
    // gate and residual of a four of tokens
    auto load_four = [&](int a) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * a + i;
            gate_r[i] = res_r[i] = 0u;
            if (kGated || !live || t >= M) continue;
            if (p.gate != nullptr) {
                const size_t gi = static_cast<size_t>(static_cast<uint32_t>(m0 + t) / p.rows_per_group) * p.N + n;
                gate_r[i] = p.gate_f32 ? static_cast<const uint32_t*>(p.gate)[gi]
                                       : static_cast<const uint16_t*>(p.gate)[gi];
            }
            if (p.res != nullptr)
                res_r[i] = reinterpret_cast<const uint16_t*>(p.res)[static_cast<size_t>(m0 + t) * p.N + n];
        }
    };
    // what the last step needs from memory, fetched while the weight streams
    auto load_epilogue = [&]() {
        load_four(first4);
        if (!live || 4 * first4 >= M) return;
        if (p.bias != nullptr) bias_r[0] = reinterpret_cast<const uint16_t*>(p.bias)[n];
        if (kGated && p.bias2 != nullptr) bias_r[1] = reinterpret_cast<const uint16_t*>(p.bias2)[n];
    };

    if (warp == 0) {
        grid_wait();
        if (lane == 0) {
            grid_launch_dependents();  // after the wait: see the head of the file
            if constexpr (!kQX) {
                for (int it = 0; it < n_first; ++it) {
                    if (it == skipped) continue;
                    load_x(it, pol);
                    if constexpr (kKind != kBf16) load_sf(C::kW, it);
                }
            }
        }
        __syncwarp();
        load_epilogue();
        if (lane == 0) {
            bool ok = true;
            int it = n_first;
            for (; it < n_stages; ++it) {
                if (!mbar_wait(&empty[it % S], ((it / S) & 1) ^ 1, kWaitNs)) {
                    ok = false;
                    break;
                }
                expect(it);
                load_w(it, pol);
                if constexpr (!kQX) load_x(it, pol);
                if constexpr (kKind != kBf16)
                    for (int o = 0; o < kSfOps; ++o) load_sf(o, it);
            }
            // every copy issued has landed before this CTA may leave or reuse its memory
            for (int i = max(0, it - S); i < it; ++i)
                if (i != skipped && !mbar_wait(&full[i % S], (i / S) & 1, kWaitNs)) ok = false;
            if (!ok) {
                record_status(MXQ_ERR_TIMEOUT);
                *failed = 1u;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        grid_wait();
        load_epilogue();
        if (lane == 0) {
            constexpr uint32_t fw = kKind == kMxf8 ? 5u : 1u;  // weight: E2M1 in both kinds
            constexpr uint32_t fx = kKind == kMxf8 ? 0u : 1u;  // activation: E4M3 / E2M1
            constexpr int kKpm = C::kKps / 4;                  // K elements an MMA
            uint32_t s = 0, ph = 0;
            bool ok = true;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!mbar_wait(kKind == kBf16 ? &full[s] : &sf_ready[s], ph, kWaitNs)) {
                    record_status(MXQ_ERR_TIMEOUT);
                    *failed = 1u;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t st = smem_u32(smem + s * C::kStage);
                const uint32_t w_lo = sdesc_sw128_lo(st), x_lo = sdesc_sw128_lo(st + C::kOffX);
                const uint32_t tsf = tmem + C::kSfCol + s * C::kSfCols;  // 32 rows of an operand to a column
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
                                    tsf + 4 * (C::kW * C::kAtoms + atom) + (m0 & 127) / 32, accum);
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
        __syncwarp();
    } else {
        grid_wait();
        load_epilogue();
        if (kKind != kBf16 && warp < 4 && lane == 0) {
            uint32_t s = 0, ph = 0;
            for (int ks = ks0; ks < ks1; ++ks) {
                // the stage's columns are free: it was refilled after its last MMAs completed
                if (!mbar_wait(&full[s], ph, kWaitNs)) {
                    record_status(MXQ_ERR_TIMEOUT);
                    *failed = 1u;
                    break;
                }
                tc_fence_after();
                const uint32_t tsf = tmem + C::kSfCol + s * C::kSfCols;
#pragma unroll
                for (int o = 0; o < C::kW + 1; ++o)
#pragma unroll
                    for (int a = 0; a < C::kAtoms && (o == C::kW) == (warp == 3); ++a)
                        tc_copy_sf_atom<1>(tsf + 4 * (o * C::kAtoms + a),
                                           sdesc_sf_atom(smem_u32(smem + C::kOffSf + (o * S + s) * C::kSf + a * 512)));
                tc_commit<1>(&sf_ready[s]);
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        if constexpr (kQX) {
            if (warp >= 4) {
                const int tid = static_cast<int>(threadIdx.x) - 128;
                QuantX<kKind> qx;
                qx.load(p, ks0, tid);
                for (int ks = ks0, it = 0; ks < ks1; ++ks, ++it) {
                    const QuantX<kKind> cur = qx;
                    if (ks + 1 < ks1) qx.load(p, ks + 1, tid);  // on its way during this stage
                    const int s = it % S;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], ((it / S) & 1) ^ 1, kWaitNs))) {
                        if (lane == 0) {
                            record_status(MXQ_ERR_TIMEOUT);
                            *failed = 1u;
                        }
                        break;
                    }
                    cur.store(p, ks, tid, smem + s * C::kStage + C::kOffX, smem + C::kOffSf + (C::kW * S + s) * C::kSf);
                    fence_async_smem();  // the tensor core reads the stage through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[s]);
                }
            }
        }
        __syncwarp();
    }
    // all MMAs are done and all copies landed
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this CTA's partials, [kW][four of tokens][128 rows][4]
    float4* part = reinterpret_cast<float4*>(smem);
    if (warp >= 4) {
        const int q = warp & 3;  // TMEM lane quarter this warp may access
#pragma unroll
        for (int w = 0; w < C::kW; ++w)
#pragma unroll 1
            for (int t0 = 0; t0 < kNT; t0 += 16) {
                if (t0 >= M) break;
                uint32_t r[16];
                tmem_ld_x16(tmem + (static_cast<uint32_t>(q * 32) << 16) + w * kNT + t0, r);
                tmem_ld_wait();
                tmem_regs_ready(r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[(w * (kNT / 4) + t0 / 4 + i) * 128 + q * 32 + lane] =
                        make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                    __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
            }
        tc_fence_before();
    }
    cluster_sync();  // the cluster's partials are written (and TMEM is read)
    tc_fence_after();
    if (warp == 1) tmem_dealloc<1>(tmem, C::kTmem);

    uint32_t bad = 0u;  // first used at the stores: the first partials are on their way before it is here
#pragma unroll
    for (int r = 0; r < kMaxSplit; ++r)
        if (r < split) bad |= ld_cluster_u32(mapa_shared(smem_u32(failed), r));
    const int fours = (M + 3) / 4;
    if (first4 >= fours) cluster_arrive();  // nothing to read from the peers
    with_act(p.act, [&](auto act) {
#pragma unroll 1
        for (int a = first4; a < fours; a += split * 2) {
            float4 v[C::kW];
#pragma unroll
            for (int w = 0; w < C::kW; ++w) {
                const uint32_t at = smem_u32(part + (w * (kNT / 4) + a) * 128 + (warp & 3) * 32 + lane);
                float4 f[kMaxSplit];
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    f[r] = r < split ? ld_cluster_f32x4(mapa_shared(at, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[w] = f[0];
#pragma unroll
                for (int r = 1; r < kMaxSplit; ++r) {
                    v[w].x += f[r].x;
                    v[w].y += f[r].y;
                    v[w].z += f[r].z;
                    v[w].w += f[r].w;
                }
            }
            // the peers may leave once the last four has been read; what follows is local
            if (a + split * 2 >= fours) cluster_arrive();
            // four tokens side by side: each step's latency is paid once for all of them
            float o[4];
            const float b0 = __uint_as_float(bias_r[0] << 16);
            const float2 lo = act_f32x2<act>(__fadd2_rn(make_float2(v[0].x, v[0].y), make_float2(b0, b0)));
            const float2 hi = act_f32x2<act>(__fadd2_rn(make_float2(v[0].z, v[0].w), make_float2(b0, b0)));
            if constexpr (kGated) {
                const float b1 = __uint_as_float(bias_r[1] << 16);
                constexpr int u = C::kW - 1;
                o[0] = lo.x * (v[u].x + b1);
                o[1] = lo.y * (v[u].y + b1);
                o[2] = hi.x * (v[u].z + b1);
                o[3] = hi.y * (v[u].w + b1);
            } else {
                const float q[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float g = p.gate == nullptr ? 1.0f : __uint_as_float(p.gate_f32 ? gate_r[i] : gate_r[i] << 16);
                    o[i] = fmaf(q[i], g, __uint_as_float(res_r[i] << 16));
                }
                if (a + split * 2 < fours) load_four(a + split * 2);
            }
            const int n_live = bad != 0u ? 0 : min(4, M - 4 * a);  // a cluster that timed out writes nothing
            const size_t row = static_cast<size_t>(m0 + 4 * a);
            if (!kGated || p.out_fmt == MXQ_OUT_BF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (live && i < n_live) p.y[(row + i) * p.N + n] = __float2bfloat16_rn(o[i]);
                continue;
            }
            if constexpr (kGated) {
                // h: the warp's 32 values of a token are one MX block (N is a multiple of 32); past N
                // they are the scale layout's padding, zeros
                const bool e4m3 = p.out_fmt == MXQ_FMT_E4M3, in = nq < p.N;
                uint32_t m[4], sc[4], code[4];
                float q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = bf16x2_bits(o[i], o[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, m[i] & 0x7FFFu);
                    sc[i] = e4m3 ? e8m0_code<8u>(top) : e8m0_code<2u>(top);
                    q[i] = lo_f(m[i]) * e8m0_inverse(sc[i]);
                }
                if (e4m3) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        code[i] = sc[i] == 255u ? 0u : cvt_e4m3x2(q[i], 0.0f);
                        if (in && i < n_live) p.q_codes[(row + i) * p.N + n] = static_cast<uint8_t>(code[i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float pair[8] = {q[i], __shfl_down_sync(0xFFFFFFFFu, q[i], 1), 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        code[i] = sc[i] == 255u ? 0u : cvt_e2m1x8(pair);
                        if (in && i < n_live && (lane & 1) == 0)
                            p.q_codes[((row + i) * p.N + n) / 2] = static_cast<uint8_t>(code[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (lane == 0 && i < n_live)
                        p.q_sf[sf_word(m0 + 4 * a + i, tile, p.atoms_n) + (warp & 3)] =
                            in ? static_cast<uint8_t>(sc[i]) : uint8_t(0);
            }
        }
    });
    // the layout's padding rows, one word of this tile each
    if (kGated && p.out_fmt != MXQ_OUT_BF16 && rank == 0 && bad == 0u && m0 + kNT >= p.M)
        for (int t = p.M + static_cast<int>(threadIdx.x); t < (p.M + 127) / 128 * 128; t += kThreads)
            *reinterpret_cast<uint32_t*>(p.q_sf + sf_word(t, tile, p.atoms_n)) = 0u;
    cluster_wait();  // no CTA leaves while another may read its partials
}

// The footprint of a few-row CTA of which one or two fit an SM, without its tensor memory: for a kernel
// that allocates it the runtime counts one CTA an SM, though here each takes at most half of it.
__global__ void __launch_bounds__(kThreads, 2) footprint_kernel() {}

// How many clusters of that many CTAs the current device holds at once, one or two CTAs an SM.  A
// property of the device (of its GPCs' sizes), asked for once.
int clusters_at_once(int split, int per_sm)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][2][kMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < kDevices)
        if (const int n = known[dev][per_sm - 1][split].load(std::memory_order_relaxed)) return n;
    const int smem = per_sm == 1 ? 227 * 1024 : 113 * 1024;
    if (cudaFuncSetAttribute(footprint_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, footprint_kernel, &cfg) != cudaSuccess) return 0;
    if (dev < kDevices) known[dev][per_sm - 1][split].store(n, std::memory_order_relaxed);
    return n;
}

// The ways K is split over a cluster.  All clusters run at once (148 SMs hold 71 of four CTAs, 45 of
// six, 37 of seven, 33 of eight; a second wave costs the whole time again: 40 tiles of 5120 x 13824
// W4A8, 48 rows, in 7 ranges 22.9 us, in 6 14.4).  A range's stages then take the longer of their round
// trip over the ring's depth and their share of the memory's rate, and CTAs that share an SM
// delay each other's set-up and last step by about 0.9 us for 16 tokens.  Measured against the
// widest split that fits: 40 tiles of K = 5120 W4A4, 48 rows, gated, in 3 11.5 us, in 6 13.4; 48
// tiles of K = 4096, one row, in 2 7.2, in 5 7.6.
int split_for(int k_stages, int64_t tiles_n, int64_t tiles_m, int stage_bytes, int ring, int nt)
{
    constexpr double kRoundTripUs = 2.0, kBytesPerUs = 6.4e6, kSharedUs = 0.9 / 16;
    const int64_t tiles = tiles_n * tiles_m;
    int best = 1;
    double best_us = 0.0;
    for (int split = 1; split <= std::min(kMaxSplit, k_stages); ++split) {
        const bool alone = tiles <= clusters_at_once(split, 1);
        if (split > 1 && !alone && tiles > clusters_at_once(split, 2)) continue;
        const double stage = std::max(kRoundTripUs / ring, static_cast<double>(tiles_n) * split * stage_bytes / kBytesPerUs);
        const double us = static_cast<double>(ceil_div(k_stages, split)) * stage + (alone ? 0.0 : kSharedUs * nt);
        if (split == 1 || us < best_us) {
            best = split;
            best_us = us;
        }
    }
    return best;
}

template <int kKind, bool kGated, int kNT, bool kQX>
cudaError_t launch_rows(const CUtensorMap (&m)[3], RowsParams& p, cudaStream_t stream)
{
    using C = Cfg<kKind, kGated, kNT>;
    const int64_t tiles_n = ceil_div(p.N, 128), tiles_m = ceil_div(p.M, kNT);
    p.split = split_for(p.k_stages, tiles_n, tiles_m, C::kTxW + C::kW * C::kSf, C::kStages, kNT);
    auto kern = gemm_rows_kernel<kKind, kGated, kNT, kQX>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(p.split * tiles_n), static_cast<unsigned>(tiles_m), 1);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, m[0], m[1], m[2], p);
}

template <int kKind, bool kGated>
cudaError_t launch_nt(int nt, const CUtensorMap (&m)[3], RowsParams& p, cudaStream_t stream)
{
    if constexpr (kKind != kBf16)
        if (p.x != nullptr) return launch_rows<kKind, kGated, 16, true>(m, p, stream);
    if (nt == 16) return launch_rows<kKind, kGated, 16, false>(m, p, stream);
    if (nt == 32) return launch_rows<kKind, kGated, 32, false>(m, p, stream);
    return launch_rows<kKind, kGated, 64, false>(m, p, stream);
}

template <int kKind>
cudaError_t launch_kind(bool gated, int nt, const CUtensorMap (&m)[3], RowsParams& p, cudaStream_t stream)
{
    return gated ? launch_nt<kKind, true>(nt, m, p, stream)
                 : launch_nt<kKind, false>(nt, m, p, stream);
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

namespace {

int num_sms()
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

}  // namespace

bool few_rows(const GemmArgs& g)
{
    if (g.M <= kRowsTileM) return true;
    const int64_t tiles = ceil_div(g.M, kRowsTileM) * ceil_div(g.N, 128);
    const bool w4a8 = !g.bf16 && g.a_fmt == kFmtE4M3;
    return tiles * (g.epilogue == kEpilogueGated ? 2 : 1) <= num_sms() * (w4a8 ? 2 : 1);
}

int launch_gemm_rows(const GemmArgs& g, cudaStream_t stream, const char** msg, char* path, size_t path_len)
{
    const bool gated = g.epilogue == kEpilogueGated;
    const int kind = g.bf16 ? kBf16 : g.a_fmt == kFmtE4M3 ? kMxf8 : kMxf4;
    const int nt = g.M <= 16 ? 16 : g.M <= 32 ? 32 : 64;
    CUtensorMap m[3];
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
    bool ok = weight(&m[0], g.w_codes);
    if (gated) ok = ok && weight(&m[1], g.w2_codes);
    else m[1] = m[0];  // never used
    const uint64_t row = kind == kMxf8 ? g.K : g.K / 2;
    if (g.x != nullptr)
        m[2] = m[0];  // never used: x is quantized inside the kernel
    else if (kind == kBf16)
        ok = ok && make_map_2d(&m[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.a_codes, g.K, g.M, g.K * 2, 64, nt,
                               CU_TENSOR_MAP_SWIZZLE_128B);
    else
        ok = ok && make_map_2d(&m[2], CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a_codes, row, g.M, row, 128, nt,
                               CU_TENSOR_MAP_SWIZZLE_128B);
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
    p.sf_w = static_cast<const uint8_t*>(g.w_sf);
    p.sf_w2 = static_cast<const uint8_t*>(g.w2_sf);
    p.sf_x = static_cast<const uint8_t*>(g.a_sf);
    p.atoms_k = static_cast<uint32_t>(sf_atoms_k(g.K));
    p.early = g.early ? 1 : 0;
    p.x = static_cast<const __nv_bfloat16*>(g.x);
    p.bias = static_cast<const __nv_bfloat16*>(g.bias);
    p.bias2 = static_cast<const __nv_bfloat16*>(g.bias2);
    p.res = static_cast<const __nv_bfloat16*>(g.residual);
    p.gate = g.gate;
    p.y = static_cast<__nv_bfloat16*>(g.y);
    p.q_codes = static_cast<uint8_t*>(g.q_codes);
    p.q_sf = static_cast<uint8_t*>(g.q_sf);

    cudaError_t e = kind == kBf16   ? launch_kind<kBf16>(gated, nt, m, p, stream)
                    : kind == kMxf8 ? launch_kind<kMxf8>(gated, nt, m, p, stream)
                                    : launch_kind<kMxf4>(gated, nt, m, p, stream);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) {
        *msg = cudaGetErrorString(e);
        return MXQ_ERR_CUDA;
    }
    if (path)
        snprintf(path, path_len, "rows%s %s 128x%d split %d tiles %d%s", g.x ? " +quantize x" : "", kind == kBf16 ? "bf16" : kind == kMxf8 ? "mxf8f6f4" : "mxf4",
                 nt, p.split, static_cast<int>(ceil_div(g.N, 128) * ceil_div(g.M, nt)), epilogue_name(g));
    return MXQ_OK;
}

}  // namespace mxq
