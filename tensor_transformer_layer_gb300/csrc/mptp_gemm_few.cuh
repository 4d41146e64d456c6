// GEMM for few tokens: C[T, N] = A[T, K] W[K, N], bound by reading W once. Tokens beyond 128 take further slices of the
// grid, which find W in L2.
//
// The roles of the operands are swapped against the large GEMM: the weight's columns are the rows of
// the product (M = 128 of them, W as stored is the MN-major operand; for W^T its rows, K-major) and the tokens its
// columns, padded to 16, so a CTA computes C^T[128, T] and a tile holds no more tokens than there are. (A 256 x 256 tile
// would multiply mostly padding, and few such tiles exist: 6 to 48 for h = 1536 or f = 6144, a part of
// the chip's 76 CTA pairs, each of which then reads a long K range alone.)
//
// The K range of a block of columns is split over the CTAs of a cluster, the largest size up to eight
// whose clusters are all resident at once. Each CTA sends its fp32 partial sums through distributed
// shared memory (four tokens a store) to the CTA that finishes those tokens, which adds them to its own in
// a fixed order: deterministic, in one launch and without a workspace.
//
//   warp 0: TMA producer, a ring of stages of 64 K rows x 128 columns (gated: 2 x 128) and the tokens' 64
//           K elements. Before it waits for the previous kernel it asks L2 for the first stages' weights.
//   warp 1: TMEM, MMA issue.   the others: partial sums out, reduction, epilogue.
//
// One token through h = 1536, f = 4096 (37.7 MB of weights): both launches 12.5 us, 38 with the large tiles; 77 tokens
// through h = 2304, f = 6144 (85 MB) 25 us. While it streams, a launch reads 7 TB/s; about 7 us go into the two
// launches' set-up, first loads and joins, and 0.07 us a token into the join.
//
// Epilogues: plain store; the gated block's gradients from dY, G and U; or gated: 128 gate columns and the 128 up columns of the same outputs have an
// accumulator each, so that a thread finds both in its TMEM lane; Y = act(gate) up is computed where the
// sums meet (GU also stored when asked for).
#pragma once

#include <atomic>

#include "mptp_gemm.cuh"
#include "mptp_internal.h"

namespace mptp {

// The weight is MN-major (its columns are the product's rows) or, transposed products, K-major (its rows are).
enum FewKind {
    FEW_PLAIN,    // C = A W
    FEW_GATED,    // Y = act(A Wg) * (A Wu), GU kept where asked for
    FEW_PLAIN_T,  // C = A W^T
    FEW_DGLU,     // dY = A W^T; dG = dY U act'(G), dU = dY act(G)
};
constexpr int FEW_SLICE = 128;   // tokens of a slice, at most
constexpr int FEW_MAX_STAGES = 8;
constexpr int FEW_MAX_PARTS = 2;  // warps of the epilogue per quarter of the tensor memory's lanes, at most
constexpr int few_threads(int parts) { return 64 + parts * 128; }
constexpr int FEW_W_BYTES = 64 * 64 * 2;  // a block of 64 K rows x 64 columns

struct FewArgs {
    int T, npad;             // tokens; tokens of a slice, a multiple of 16
    int blocks;              // blocks of 128 columns
    int kb;                  // K blocks of 64
    int cols;                // output columns (gated: f)
    int w_cols;              // columns of W
    int up_off;              // gated: columns of W from a gate to its up
    int cluster, stages;
    int parts;               // warps of the epilogue a quarter of the lanes: shares of the tokens
    int act;
    __nv_bfloat16* out;      // [T, cols]; dGLU: [T, 2 cols]
    __nv_bfloat16* gu;       // [T, 2 cols]; gated, nullable: written; dGLU: read
    uint32_t* status;
    unsigned long long budget_ns;
};

__host__ __device__ inline size_t few_stage_bytes(bool gated, int npad) { return (gated ? 4 : 2) * FEW_W_BYTES + size_t(npad) * 128; }
// Tokens that each CTA of a cluster finishes: whole groups of four.
__host__ __device__ inline int few_slice(int npad, int cluster) { return (npad / 4 + cluster - 1) / cluster * 4; }
// Partial sums that a CTA receives: from every rank, its slice's tokens x 128 columns (x 2, gated).
__host__ __device__ inline size_t few_red_bytes(bool gated, int npad, int cluster) {
    return size_t(cluster) * few_slice(npad, cluster) * 128 * 4 * (gated ? 2 : 1);
}
// The partial sums take the ring's place once every CTA of the cluster has used its stages.
__host__ __device__ inline size_t few_ring_bytes(bool gated, int npad, int cluster, int stages) {
    const size_t ring = stages * few_stage_bytes(gated, npad), red = few_red_bytes(gated, npad, cluster);
    return ring > red ? ring : red;
}
inline size_t few_smem_bytes(bool gated, int npad, int cluster, int stages) {
    return 1024 + few_ring_bytes(gated, npad, cluster, stages) + 8 * (2 * FEW_MAX_STAGES + 2) + 16;
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}

// Bounded wait whose probes do not suspend the thread, so that any budget is kept to, one below a probe's longest
// suspension too. For the one wait of the epilogue's warps: the whole K range's time.
__device__ __forceinline__ bool wait_polled(uint64_t* bar, uint32_t parity, const Ctl& c) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_test_wait(bar, parity)) return true;
        if (*c.abort_flag) return false;
        if (globaltimer_ns() - t0 > c.budget_ns) {
            if (c.status) atomicOr(c.status, DEV_TIMEOUT);
            *c.abort_flag = 1u;
            return false;
        }
    }
}

template <int KIND>
__global__ void __launch_bounds__(few_threads(FEW_MAX_PARTS)) gemm_few_kernel(const __grid_constant__ CUtensorMap tmW,
                                                               const __grid_constant__ CUtensorMap tmA,
                                                               const FewArgs args) {
    constexpr bool GATED = KIND == FEW_GATED, W_T = KIND == FEW_PLAIN_T || KIND == FEW_DGLU;
    constexpr int NACC = GATED ? 2 : 1;            // accumulators: gate and up
    constexpr int W_STAGE = 2 * NACC * FEW_W_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int npad = args.npad, stages = args.stages, cluster = args.cluster;
    const int slice = few_slice(npad, cluster);
    uint8_t* sW = smem;                            // stage s at s * W_STAGE
    uint8_t* sA = smem + stages * W_STAGE;         // stage s at s * npad * 128
    // [source rank][four tokens of the slice][accumulator][128 columns] x 4 tokens
    float4* red = reinterpret_cast<float4*>(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + few_ring_bytes(GATED, npad, cluster, stages));
    uint64_t* full = bars;
    uint64_t* empty = bars + FEW_MAX_STAGES;
    uint64_t* acc_full = bars + 2 * FEW_MAX_STAGES;
    uint64_t* drain_bar = acc_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int block = static_cast<int>(blockIdx.x) / cluster % args.blocks;
    const int t0 = static_cast<int>(blockIdx.x) / cluster / args.blocks * npad;  // first token of the slice
    const int T = min(npad, args.T - t0);
    const int kb0 = args.kb * rank / cluster, kb1 = args.kb * (rank + 1) / cluster;
    const uint32_t need_cols = NACC * npad;
    const uint32_t tmem_cols = need_cols <= 32 ? 32u : need_cols <= 64 ? 64u : need_cols <= 128 ? 128u : 256u;

    // Weight columns of the stage's i-th 64-wide block. A last block behind the columns reads zeros (or,
    // gated, columns of the ups, whose results are not stored).
    auto w_col = [&](int i) { return block * 128 + (i & 1) * 64 + (i >> 1) * args.up_off; };
    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmA);
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        // Into L2 only: whatever the previous kernel may still write is read after the wait below.
        for (int kb = kb0; kb < kb1 && kb < kb0 + stages; ++kb)
            if constexpr (W_T) {
                tma_prefetch_2d(&tmW, kb * BK, block * 128);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * NACC; ++i)
                    if (w_col(i) < args.w_cols) tma_prefetch_2d(&tmW, w_col(i), kb * BK);
            }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Ctl ctl{args.status, abort_flag, args.budget_ns};
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == 0) {
        // A wait budget of zero stands for loads that never arrive, of a cluster's in its last CTA.
        if (lane == 0 && !(args.budget_ns == 0 && rank == cluster - 1)) {
            int st = 0;
            uint32_t ph = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bounded(&empty[st], ph ^ 1u, ctl)) break;
                mbar_arrive_expect_tx(&full[st], W_STAGE + npad * 128);
                if constexpr (W_T) {
                    tma_load_2d(sW + st * W_STAGE, &tmW, &full[st], kb * BK, block * 128);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * NACC; ++i)
                        tma_load_2d(sW + st * W_STAGE + i * FEW_W_BYTES, &tmW, &full[st], w_col(i), kb * BK);
                }
                tma_load_2d(sA + st * npad * 128, &tmA, &full[st], kb * BK, t0);
                if (++st == stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = make_idesc_bf16(128, npad, !W_T, false);
        const uint64_t w_desc = make_sdesc_sw128(smem_u32(sW), W_T ? 16 : FEW_W_BYTES, 1024);
        constexpr int W_STEP = W_T ? 32 : 2048;  // bytes from one product's rows of K to the next's
        const uint64_t a_desc = make_sdesc_sw128(smem_u32(sA), 16, 1024);
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
            const bool got = wait_bounded(&full[st], ph, ctl);
            if (!(ok = __all_sync(0xffffffffu, got) != 0)) break;
            tc_fence_after();
            const uint64_t wd = w_desc + static_cast<uint32_t>((st * W_STAGE) >> 4);
            const uint64_t ad = a_desc + static_cast<uint32_t>((st * npad * 128) >> 4);
#pragma unroll
            for (int k = 0; k < BK / UMMA_K; ++k)
#pragma unroll
                for (int c = 0; c < NACC; ++c)
                    umma_bf16_elect(tmem_base + c * npad, wd + c * (2 * FEW_W_BYTES >> 4) + k * (W_STEP >> 4),
                                    ad + k * (32 >> 4), idesc, kb > kb0 || k > 0 ? 1u : 0u);
            umma_commit_elect(&empty[st]);
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        if (ok) umma_commit_elect(acc_full);
        umma_commit_elect(drain_bar);
        wait_drain(drain_bar, 0, args.status);
    }
    const int q = warp & 3;
    const int part = (warp - 2) >> 2, parts = args.parts;
    const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const int col = q * 32 + lane;  // column of the block
    bool got = true;
    if (warp >= 2) {
        got = wait_polled(acc_full, 0, ctl);
        got = __all_sync(0xffffffffu, got) != 0;
    }
    __syncwarp();
    if (cluster > 1) cluster_sync_all();  // every CTA of the cluster has used its ring: it may be written over
    if (warp >= 2) {
        // This CTA's partial sums, four tokens at a time, to the CTAs that finish them; its own tokens' stay.
        if (got) {
            tc_fence_after();
#pragma unroll 1
            for (int c = part * 16; c < T && cluster > 1; c += parts * 16) {
                uint32_t v[NACC][16];
#pragma unroll
                for (int i = 0; i < NACC; ++i) tmem_ld16(t_addr + i * npad + c, v[i]);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < NACC; ++i) reg_fence16(v[i]);
                int owner = c / slice, at = (c - owner * slice) / 4;  // the four tokens' CTA, and their place there
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (c + 4 * g < T && owner != rank) {
                        float4* dst = red + ((rank * (slice / 4) + at) * NACC) * 128 + col;
                        const uint32_t to = mapa_shared(smem_u32(dst), owner);
#pragma unroll
                        for (int i = 0; i < NACC; ++i)
                            st_cluster_v4(to + i * 2048, v[i][4 * g], v[i][4 * g + 1], v[i][4 * g + 2], v[i][4 * g + 3]);
                    }
                    if (++at == slice / 4) {
                        at = 0;
                        ++owner;
                    }
                }
            }
        }
    } else if (warp == 0 && lane < cluster && cluster > 1 && *abort_flag != 0u) {
        // This CTA gave up and sends nothing: the others would add old stages in its place. They give up too.
        st_cluster_b32(mapa_shared(smem_u32(const_cast<uint32_t*>(abort_flag)), lane), 1u);
    }
    __syncwarp();
    if (cluster > 1)
        cluster_sync_all();  // releases the partial sums, acquires the others'
    else
        __syncthreads();
    if (warp >= 2 && *abort_flag == 0u && block * 128 + q * 32 < args.cols) {
        // Eight tokens of a column at a time: their loads, then their arithmetic, then their stores. (Four at a time,
        // through pointers that the stores might alias, took 800 cycles each.)
        constexpr int G = 2;
        const int c0 = rank * slice, c1 = min(T, c0 + slice);
#pragma unroll 1
        for (int c = c0 + part * 4 * G; c < c1; c += parts * 4 * G) {
            float gate[G * 4], up[G * 4];
            if constexpr (KIND == FEW_DGLU) {
                const __nv_bfloat16* gu = args.gu + static_cast<long long>(t0 + c) * 2 * args.cols + block * 128 + col;
#pragma unroll
                for (int k = 0; k < G * 4; ++k, gu += 2 * args.cols) {
                    gate[k] = c + k < c1 ? __bfloat162float(gu[0]) : 0.0f;
                    up[k] = c + k < c1 ? __bfloat162float(gu[args.cols]) : 0.0f;
                }
            }
            uint32_t own[G][NACC][4];
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (g == 0 || c + 4 * g < c1)
#pragma unroll
                    for (int i = 0; i < NACC; ++i) tmem_ld4(t_addr + i * npad + c + 4 * g, own[g][i]);
            tmem_wait_ld();
            float sum[G][NACC][4];
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < NACC; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        asm volatile("" : "+r"(own[g][i][e]));
                        sum[g][i][e] = __uint_as_float(own[g][i][e]);
                    }
            // own first, then the ranks behind it in turn: a fixed order for every token
#pragma unroll 2
            for (int s = 1; s < cluster; ++s) {
                const int from = rank + s - (rank + s >= cluster ? cluster : 0);
                const uint32_t at = smem_u32(red) + (((from * slice + c - c0) / 4 * NACC) * 128 + col) * 16;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    if (g == 0 || c + 4 * g < c1)
#pragma unroll
                        for (int i = 0; i < NACC; ++i) {
                            const float4 v = ld_shared_v4(at + (g * NACC + i) * 2048);
                            sum[g][i][0] += v.x;
                            sum[g][i][1] += v.y;
                            sum[g][i][2] += v.z;
                            sum[g][i][3] += v.w;
                        }
            }
            if constexpr (KIND == FEW_DGLU) {
                __nv_bfloat16* out = args.out + static_cast<long long>(t0 + c) * 2 * args.cols + block * 128 + col;
#pragma unroll
                for (int k = 0; k < G * 4; k += 2, out += 4 * args.cols) {
                    const float2 dy = make_float2(sum[k / 4][0][k % 4], sum[k / 4][0][k % 4 + 1]);
                    float2 act, slope;
                    glu_act_grad2(make_float2(gate[k], gate[k + 1]), args.act, act, slope);
                    const float2 dg = mul2(mul2(dy, make_float2(up[k], up[k + 1])), slope), du = mul2(dy, act);
                    if (c + k < c1) {
                        out[0] = __float2bfloat16(dg.x);
                        out[args.cols] = __float2bfloat16(du.x);
                    }
                    if (c + k + 1 < c1) {
                        out[2 * args.cols] = __float2bfloat16(dg.y);
                        out[3 * args.cols] = __float2bfloat16(du.y);
                    }
                }
            } else {
                float y[G * 4];
#pragma unroll
                for (int k = 0; k < G * 4; k += 2) {
                    float2 v = make_float2(sum[k / 4][0][k % 4], sum[k / 4][0][k % 4 + 1]);
                    if constexpr (GATED)
                        v = mul2(glu_act2(v, args.act), make_float2(sum[k / 4][1][k % 4], sum[k / 4][1][k % 4 + 1]));
                    y[k] = v.x, y[k + 1] = v.y;
                }
                __nv_bfloat16* out = args.out + static_cast<long long>(t0 + c) * args.cols + block * 128 + col;
#pragma unroll
                for (int k = 0; k < G * 4; ++k, out += args.cols)
                    if (c + k < c1) *out = __float2bfloat16(y[k]);
                if constexpr (GATED)
                    if (args.gu) {
                        __nv_bfloat16* gu = args.gu + static_cast<long long>(t0 + c) * 2 * args.cols + block * 128 + col;
#pragma unroll
                        for (int k = 0; k < G * 4; ++k, gu += 2 * args.cols)
                            if (c + k < c1) {
                                gu[0] = __float2bfloat16(sum[k / 4][0][k % 4]);
                                gu[args.cols] = __float2bfloat16(sum[k / 4][1][k % 4]);
                            }
                    }
            }
        }
    }

    // ---------------- teardown ----------------
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        if (threadIdx.x == 0) spin_ns(ABORT_SETTLE_NS);
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// Clusters of `cluster` CTAs of this kernel that are resident at once.
template <int KIND>
inline int few_resident_clusters(int cluster, size_t smem, int num_sms) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster * num_sms, 1, 1);
    cfg.blockDim = dim3(few_threads(FEW_MAX_PARTS), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, gemm_few_kernel<KIND>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// C[T, cols] = A[T, K] W[K, ...], or A W^T with W [cols, K]; W's rows are `ldw` columns wide.
template <int KIND>
inline mp_status launch_gemm_few(const mp_bf16* A, const mp_bf16* W, mp_bf16* out, mp_bf16* gu, int T, int K, int cols,
                                 int ldw, int act, uint32_t* status, int num_sms, cudaStream_t stream) {
    constexpr bool GATED = KIND == FEW_GATED, W_T = KIND == FEW_PLAIN_T || KIND == FEW_DGLU;
    FewArgs a{};
    a.T = T;
    a.blocks = ceil_div(cols, 128);
    // Slices of tokens: as few as hold them all, then halves while clusters of some CTAs remain for each: the join of
    // the partial sums grows with a slice's tokens and is the longer part where the weights are few. Measured for the
    // whole block, 128 tokens, without and with halves: h = 1024, f = 2048 18.5 and 13.3 us, h = 1536, f = 4096 21.5
    // and 18.1, h = 2304, f = 6144 28.7 and 27.7. Smaller slices, or smaller clusters, lose: the plain product's halves
    // at clusters of two take 24.4 us against 21.9 for 256 tokens, h = 1536.
    constexpr int LEAST = GATED ? 32 : 64, LEAST_CLUSTER = GATED ? 2 : 4;
    int slices = ceil_div(T, FEW_SLICE);
    while (ceil_div(T, 2 * slices) >= LEAST && a.blocks * 2 * slices * LEAST_CLUSTER <= num_sms) slices *= 2;
    a.npad = ceil_div(ceil_div(T, slices), 16) * 16;
    a.kb = K / BK;
    a.cols = cols;
    a.w_cols = ldw;
    a.up_off = cols;
    a.act = act;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.gu = reinterpret_cast<__nv_bfloat16*>(gu);
    a.status = status;
    a.budget_ns = wait_budget_ns();
    CUtensorMap tw, ta;
    if (!(W_T ? make_tmap_bf16(&tw, W, K, cols, ldw, 64, 128) : make_tmap_bf16(&tw, W, ldw, K, ldw, 64, 64)) ||
        !make_tmap_bf16(&ta, A, K, T, K, 64, a.npad))
        return MP_ERR_CUDA;
    auto kern = gemm_few_kernel<KIND>;
    const int clusters = a.blocks * slices;
    auto fit_stages = [&](int cluster) {
        int n = FEW_MAX_STAGES;
        while (few_smem_bytes(GATED, a.npad, cluster, n) > SMEM_LIMIT) --n;
        return n;
    };
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_LIMIT)) != cudaSuccess)
        return MP_ERR_CUDA;
    // How many clusters of a size are resident depends on the device alone (one CTA an SM): looked up once.
    static std::atomic<int> cached[16][9];
    int dev = 0;
    cudaGetDevice(&dev);
    a.cluster = 1;
    for (int c = 8; c > 1; --c) {
        if (a.kb < 2 * c) continue;
        std::atomic<int>* slot = dev < 16 ? &cached[dev][c] : nullptr;
        int n = slot ? slot->load(std::memory_order_relaxed) : 0;
        if (n == 0) {
            n = few_resident_clusters<KIND>(c, SMEM_LIMIT, num_sms);
            if (slot) slot->store(n > 0 ? n : -1, std::memory_order_relaxed);
        }
        if (clusters <= n) {
            a.cluster = c;
            break;
        }
    }
    a.stages = fit_stages(a.cluster);
    // Eight warps finish the tokens where there are more than a few: 77 tokens, h = 2304, f = 6144 24.9 us against 26.1
    // with four, one token 21.1 against 20.7. (Sixteen: 25.6 and 22.0.)
    a.parts = T <= 32 ? 1 : FEW_MAX_PARTS;
    const size_t smem = few_smem_bytes(GATED, a.npad, a.cluster, a.stages);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(clusters * a.cluster);
    cfg.blockDim = dim3(few_threads(a.parts));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tw, ta, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

}  // namespace mptp
