// Entry point of the packed attention's backward: mp_attn_varlen_bwd.
//
//   P = exp(scale Q K^T - LSE)          recomputed tile by tile, never stored
//   delta = rowsum(dO * O)
//   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q
//
// Two kernels, each with its own recomputation of S and dP: one walks a query tile's keys and keeps
// dQ in tensor memory, the other walks a key tile's queries and keeps dK and dV there. That is seven
// products per pair of tiles where five would do, but no gradient is summed across CTAs: no atomics,
// no fp32 gradient in memory, a fixed order and so the same bits every run. (One kernel with five
// products would also be bound by shared memory: at D = 128 its dS goes through it once more and 64 KB
// of fp32 dQ per pair of tiles leave through it, against 64 KB a tile of K or Q loads for each here. That is an estimate
// for D = 128; at D = 64, where both kernels wait for the same softmax, one kernel has not been measured.)
//
// dQ kernel: CTA = (sequence, query head, 128 queries). Per key tile S = Q K^T, dP = dO V^T and
//   dQ += dS K with dS (bf16) read from tensor memory. S has two buffers and is computed two tiles ahead,
//   so the softmax warps go from dS(j) to S(j+1) at once. The CTA first computes its rows' delta and leaves it for the
//   other kernel. Where a single key tile holds all that the rows see, delta is summed as P dP instead,
//   which is the same without O's rounding to bf16: rows of few keys sit there, whose O is large and whose
//   dP - delta cancels most (two keys, D = 128: dQ's error 8.0e-3 of its norm from O, 2.6e-3 from P dP).
// dK, dV kernel: CTA = (sequence, key head, 128 keys), over the queries of every head of the group (so
//   shared key heads need no sum across CTAs either). Scores are computed transposed, S^T = K Q^T and
//   dP^T = V dO^T, one key per TMEM lane: P^T and dS^T are then A operands in tensor memory as they
//   stand, dV += P^T dO and dK += dS^T Q, and dO and Q serve as loaded (MN-major). At D = 128 the four
//   accumulators take all 512 columns: P^T lies over S^T, so S(i+1) follows dV(i), and the products of one
//   half of the softmax (dV, S) run while the warps are at the other half (dK, dP). At D <= 96 there is room
//   for a second S^T or for P^T beside it: S^T runs ahead and the warps never wait for it.
//   Where whole key tiles would balance badly (few of them, many queries each), a cluster of two to eight CTAs
//   shares one: each takes a part of its (head, query tile) pairs, and the fp32 sums are joined through
//   distributed shared memory in rank order. The dQ kernel shares a query tile's keys the same way.
// In the first, a softmax thread has one row and 64 of its 128 columns; in the second, four keys' fragments.
// Both are bound by the hand-overs between softmax and products (tensor core 65 to 67 % active at D = 128): 4096
// tokens, 19 heads, not causal, dQ 114, 134, 158 us and dK with dV 139, 180, 210 us for D = 64, 96, 128 (1.07 to 1.55
// and 1.17 to 1.55 PFLOP/s). The warp that issues the products is on the way between them: rings counted along instead
// of remainders, and no clearing between a wait and a product, took dQ from 139 and 166 us at D = 96 and 128. Sixteen softmax warps of half the columns each were 1 to 10 % slower.
//
// P and dS are rounded to bf16 for their products (the tensor core's operand type; with the results' own rounding, dQ,
// dK and dV are 2.4e-3 of their norm off, the results of fp32 products rounded once 1.7e-3); the exponent,
// delta, and every sum are fp32. Hidden pairs' dS (for dQ) and P (for dV, and through it dS for dK) are replaced by zero
// after the arithmetic; rows of a tile behind the sequence's end are cleared in shared memory where they would be summed
// over, and queries that see no key are not loaded.
#include <type_traits>

#include "mptp_attn_varlen.cuh"

namespace mptp {

__device__ __forceinline__ void softmax_warps_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A row's log-sum-exp in exp2 units, +inf (every probability 0) where it saw no key.
__device__ __forceinline__ float lse_to_log2(float lse) {
    return lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
}

// ------------------------------------------------------------------------------------------------
// dQ (and delta)
// ------------------------------------------------------------------------------------------------
template <int D>
struct AvDqCfg {
    using T = AvTile<D>;
    static constexpr int KST = D == 128 ? 3 : 4;  // a K tile serves S(j) and, later, dQ(j)
    static constexpr int VST = D == 64 ? 4 : D == 96 ? 3 : 2;
    static constexpr int NUM_BARS = 2 + 2 * KST + 2 * VST + 2 + 4 + 1;
    static constexpr size_t SMEM = 1024 + (2 + KST + VST) * size_t(T::BYTES) + 2 * AV_TILE * 4 + 8 * NUM_BARS + 16;
    static_assert(SMEM <= SMEM_LIMIT, "shared memory per block");
    static_assert((KST + VST) * T::BYTES >= 8 * AV_TILE * 128, "a chunk of every part at the join");
    static constexpr uint32_t TMEM_COLS = 512;  // S(even), S(odd) at 0, 128; dP at 256; dQ at 384
};

template <int D, bool JOIN>
__global__ void __launch_bounds__(AV_THREADS, 1)
    attn_varlen_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                          const __grid_constant__ CUtensorMap tmdQ, const __nv_bfloat16* O, long long ldo,
                          const __nv_bfloat16* dO, long long lddo, const float* LSE, float* delta, __nv_bfloat16* dQ,
                          long long lddq, int cluster_size, const AvArgs args) {
    const int cluster = JOIN ? cluster_size : 1;
    using Cfg = AvDqCfg<D>;
    using T = AvTile<D>;
    constexpr int NB = T::NB, KST = Cfg::KST, VST = Cfg::VST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sdO = sQ + T::BYTES;
    uint8_t* sK = sdO + T::BYTES;
    uint8_t* sV = sK + KST * T::BYTES;
    float* part = reinterpret_cast<float*>(sV + VST * T::BYTES);  // [2][128] halves of delta
    uint64_t* bars = reinterpret_cast<uint64_t*>(part + 2 * AV_TILE);
    uint64_t* q_full = bars;
    uint64_t* do_full = bars + 1;
    uint64_t* k_full = bars + 2;
    uint64_t* k_empty = k_full + KST;
    uint64_t* v_full = k_empty + KST;
    uint64_t* v_empty = v_full + VST;
    uint64_t* s_full = v_empty + VST;  // [2]
    uint64_t* dp_full = s_full + 2;
    uint64_t* ds_full = dp_full + 1;   // dS(j) is in tensor memory
    uint64_t* dq_full = ds_full + 1;
    uint64_t* part_full = dq_full + 1; // both halves of delta from one key tile
    uint64_t* drain_bar = part_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int item = static_cast<int>(blockIdx.x) / cluster;
    const int rank = JOIN ? static_cast<int>(cluster_ctarank()) : 0;
    const int head = item % args.heads;
    const int kvh = head / args.group;

    grid_dependency_wait();
    AvSpan sp;
    int qt;
    if (!av_pick<AV_TILE, true>(args, item / args.heads, sp, qt))
        return;
    const int i0 = qt * AV_TILE;
    const int n_all = av_key_tiles(sp, i0, args.causal);
    // this CTA's part of the key tiles
    auto part_begin = [&](int r) { return n_all * r / cluster; };
    const int n = part_begin(rank + 1) - part_begin(rank);
    const int kb = part_begin(rank) * AV_TILE, k_row = sp.k0 + kb;
    const int k_tail = n * AV_TILE > sp.nk - kb ? sp.nk - kb - (n - 1) * AV_TILE : AV_TILE;

    // The softmax warps' rows of LSE, O and dO are asked for before the set-up, which takes as long as they do.
    // delta = rowsum(dO * O): each warp sums 16 rows, whole rows side by side, 16 bytes a lane. (Row by row, a row
    // to a thread, they took 8000 cycles at D = 96: the shared memory leaves no cache to hold a line for the next
    // piece.) With one key tile the loop sums delta instead.
    const bool one_tile = n_all == 1;
    constexpr int LANES = D / 8, ROWS = 32 / LANES, LOADS = 16 / ROWS;  // lanes a row, rows a load, loads a warp
    uint4 o_part[LOADS], do_part[LOADS];
    const long long row_at = static_cast<long long>(head) * args.Tq + sp.q0 + i0 + (warp & 3) * 32 + lane;
    float lse = -INFINITY;
    if (warp >= 4) {
        if (i0 + (warp & 3) * 32 + lane < sp.nq) lse = LSE[row_at];
        if (!one_tile) {
#pragma unroll
            for (int u = 0; u < LOADS; ++u) {
                const int m = (warp - 4) * 16 + u * ROWS + lane / LANES;
                o_part[u] = do_part[u] = make_uint4(0u, 0u, 0u, 0u);
                if (lane / LANES < ROWS && i0 + m < sp.nq) {
                    const long long at = sp.q0 + i0 + m;
                    const int c = head * D + lane % LANES * 8;
                    o_part[u] = *reinterpret_cast<const uint4*>(O + at * ldo + c);
                    do_part[u] = *reinterpret_cast<const uint4*>(dO + at * lddo + c);
                }
            }
        }
    }

    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(do_full, 1);
        for (int i = 0; i < KST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VST; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1);
        mbar_init(ds_full, 8);
        mbar_init(dq_full, 1);
        mbar_init(part_full, 8);
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        if (n > 0 && !av_starved(args, rank, cluster)) {
            av_load<D>(sK, &tmK, &k_full[0], kvh, k_row);
            av_load<D>(sQ, &tmQ, q_full, head, sp.q0 + i0);
            av_load<D>(sV, &tmV, &v_full[0], kvh, k_row);
            av_load<D>(sdO, &tmdO, do_full, head, sp.q0 + i0);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_launch_dependents();  // once this CTA holds its tensor memory: a dependent may want some too
    const Ctl ctl{args.status, abort_flag, args.budget_ns};
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool got = wait_bounded(bar, parity, ctl);
        return __all_sync(0xffffffffu, got) != 0;
    };

    if (warp < 4) {
        reg_dealloc<T::REGS_CTRL>();
        if (warp == 0) {
            if (lane == 0) {
                // ---------------- TMA producer ----------------
                bool ok = true;
                for (int j = 1; j < n && ok; ++j) {
                    int st = j % KST;
                    ok = wait_bounded(&k_empty[st], ((j / KST) & 1) ^ 1u, ctl);
                    if (!ok) break;
                    av_load<D>(sK + st * T::BYTES, &tmK, &k_full[st], kvh, k_row + j * AV_TILE);
                    st = j % VST;
                    ok = wait_bounded(&v_empty[st], ((j / VST) & 1) ^ 1u, ctl);
                    if (!ok) break;
                    av_load<D>(sV + st * T::BYTES, &tmV, &v_full[st], kvh, k_row + j * AV_TILE);
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            constexpr uint32_t IDESC_S = make_idesc_bf16(AV_TILE, AV_TILE, false, false);
            constexpr uint32_t IDESC_DQ = make_idesc_bf16(AV_TILE, D, false, true);
            const uint64_t q_desc = make_sdesc_sw64(smem_u32(sQ), 16, 512);
            const uint64_t do_desc = make_sdesc_sw64(smem_u32(sdO), 16, 512);
            const uint64_t k_desc = make_sdesc_sw64(smem_u32(sK), 16, 512);
            const uint64_t kt_desc = make_sdesc_sw64(smem_u32(sK), T::BOX, 512);  // keys summed over
            const uint64_t v_desc = make_sdesc_sw64(smem_u32(sV), 16, 512);
            auto score = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 1) * T::BOX + (k & 1) * 32) >> 4;
                    umma_bf16_elect(d, a + off, b + off, IDESC_S, k > 0 ? 1u : 0u);
                }
            };
            AvRing<KST> k_next, k_sum;  // K tiles of the next S and of the next dQ
            AvRing<VST> v_next;
            auto k_wait = [&]() { return wait_all(&k_full[k_next.st], k_next.ph); };
            auto v_wait = [&]() { return wait_all(&v_full[v_next.st], v_next.ph); };
            auto s_mma = [&](int buf) {
                score(tmem_base + buf * 128, q_desc, k_desc + static_cast<uint32_t>((k_next.st * T::BYTES) >> 4));
                umma_commit_elect(&s_full[buf]);
                k_next.next();
            };
            auto dp_mma = [&]() {
                score(tmem_base + 256, do_desc, v_desc + static_cast<uint32_t>((v_next.st * T::BYTES) >> 4));
                umma_commit_elect(dp_full);
                umma_commit_elect(&v_empty[v_next.st]);
                v_next.next();
            };
            bool ok = n > 0 && wait_all(q_full, 0) && k_wait();
            if (ok) {
                tc_fence_after();
                s_mma(0);
                ok = wait_all(do_full, 0) && v_wait();
                if (ok) {
                    tc_fence_after();
                    dp_mma();
                }
            }
            // One wait on the softmax an iteration, and three products behind it: dP(j+1), which it needs next,
            // dQ(j), and S(j+2) over dS(j) once that has been used. (With a wait before each of the products the
            // tensor core ran dry at every one: 2140 cycles an iteration at D = 128, 1536 of them products.)
            if (ok && n > 1 && (ok = k_wait())) {
                tc_fence_after();
                s_mma(1);
            }
            for (int j = 0; j < n && ok; ++j) {
                const bool more = j + 1 < n, ahead = j + 2 < n;
                if (more && !(ok = v_wait())) break;
                // The foreign rows of the last key tile, which dQ sums over: S needs no clearing, its columns are masked.
                if (!more && k_tail < AV_TILE) av_clear_rows<D>(sK + k_sum.st * T::BYTES, k_tail, lane);
                if (!(ok = wait_all(ds_full, j & 1))) break;
                tc_fence_after();
                if (more) dp_mma();
                const uint64_t kd = kt_desc + static_cast<uint32_t>((k_sum.st * T::BYTES) >> 4);
                const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
                for (int k = 0; k < AV_TILE / 16; ++k)
                    umma_bf16_ts_elect(tmem_base + 384, av_a_step(tmem_base + (j & 1) * 128, k), kd + ((k * 1024) >> 4),
                                       IDESC_DQ, k > 0 ? 1u : acc0);
                umma_commit_elect(&k_empty[k_sum.st]);
                k_sum.next();
                if (ahead) {
                    if (!(ok = k_wait())) break;
                    tc_fence_after();
                    s_mma(j & 1);
                }
            }
            if (ok) umma_commit_elect(dq_full);
            umma_commit_elect(drain_bar);
            wait_drain(drain_bar, 0, args.status);
        }
    } else {
        reg_alloc<T::REGS_SOFTMAX>();
        // ---------------- softmax: warps 4..7 key columns 0..63, warps 8..11 columns 64..127 ----------------
        const int hf = (warp - 4) >> 2;
        const int q = warp & 3;
        const int w0 = i0 + q * 32;
        const int qi = w0 + lane;
        const int rows_ok = min(32, sp.nq - w0);
        const bool row_ok = lane < rows_ok;
        float dl = 0.0f;
        if (!one_tile) {
#pragma unroll
            for (int u = 0; u < LOADS; ++u) {
                const uint32_t aw[4] = {o_part[u].x, o_part[u].y, o_part[u].z, o_part[u].w};
                const uint32_t bw[4] = {do_part[u].x, do_part[u].y, do_part[u].z, do_part[u].w};
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sum = fmaf(bf16_lo(aw[k]), bf16_lo(bw[k]), sum);
                    sum = fmaf(bf16_hi(aw[k]), bf16_hi(bw[k]), sum);
                }
                // the row's lanes, in a fixed order: its first lane ends with the sum
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    const float v = __shfl_down_sync(0xffffffffu, sum, o);
                    if (lane % LANES + o < LANES) sum += v;
                }
                if (lane / LANES < ROWS && lane % LANES == 0) part[(warp - 4) * 16 + u * ROWS + lane / LANES] = sum;
            }
            softmax_warps_sync();  // no warp has left: there was no wait before it
            dl = part[q * 32 + lane];
        }
        const float lse2 = lse_to_log2(lse);
        const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_addr + hf * 64;
        const uint32_t dp_addr = tmem_base + lane_addr + 256 + hf * 64;
        const int off = sp.nk - sp.nq;
        const int see = (args.causal ? min(sp.nk, qi + off + 1) : sp.nk) - kb;
        const int see_w = (args.causal ? min(sp.nk, w0 + off + 1) : sp.nk) - kb;
        const float2 c2v = make_float2(args.scale_log2, args.scale_log2);
        const float2 nl = make_float2(-lse2, -lse2);
        bool ok = true;
        for (int j = 0; j < n && ok; ++j) {
            const uint32_t s_buf = s_addr + (j & 1) * 128;
            if (!(ok = wait_all(&s_full[j & 1], (j >> 1) & 1))) break;
            tc_fence_after();
            uint32_t p[2][32];
            tmem_ld32(s_buf, p[0]);
            tmem_ld32(s_buf + 32, p[1]);
            tmem_wait_ld();
            reg_fence32(p[0]);
            reg_fence32(p[1]);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                uint32_t& a = p[(2 * k) >> 5][(2 * k) & 31];
                uint32_t& b = p[(2 * k + 1) >> 5][(2 * k + 1) & 31];
                const float2 x = fma2(make_float2(__uint_as_float(a), __uint_as_float(b)), c2v, nl);
                a = __float_as_uint(ex2_approx(x.x));
                b = __float_as_uint(ex2_approx(x.y));
            }
            if (!(ok = wait_all(dp_full, j & 1))) break;
            tc_fence_after();
            uint32_t t[2][32];
            tmem_ld32(dp_addr, t[0]);
            tmem_ld32(dp_addr + 32, t[1]);
            tmem_wait_ld();
            reg_fence32(t[0]);
            reg_fence32(t[1]);
            uint32_t w[32];
            const int lim = see - j * AV_TILE - hf * 64;  // visible columns of this thread
            if (one_tile) {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    const float v = __uint_as_float(p[k >> 5][k & 31]) * __uint_as_float(t[k >> 5][k & 31]);
                    sum += k < lim ? v : 0.0f;
                }
                part[hf * AV_TILE + q * 32 + lane] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(part_full);
                if (!(ok = wait_all(part_full, 0))) break;
                dl = part[q * 32 + lane] + part[AV_TILE + q * 32 + lane];
            }
            const float2 nd = make_float2(-dl, -dl);
            auto grad = [&](auto masked) {
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float2 pr = make_float2(__uint_as_float(p[(2 * k) >> 5][(2 * k) & 31]),
                                                  __uint_as_float(p[(2 * k + 1) >> 5][(2 * k + 1) & 31]));
                    const float2 dp = make_float2(__uint_as_float(t[(2 * k) >> 5][(2 * k) & 31]),
                                                  __uint_as_float(t[(2 * k + 1) >> 5][(2 * k + 1) & 31]));
                    float2 ds = mul2(pr, add2(dp, nd));
                    if (decltype(masked)::value) {
                        ds.x = 2 * k < lim ? ds.x : 0.0f;
                        ds.y = 2 * k + 1 < lim ? ds.y : 0.0f;
                    }
                    w[k] = pack_bf16x2(ds.x, ds.y);
                }
            };
            if (see_w < j * AV_TILE + hf * 64 + 64)
                grad(std::true_type{});
            else
                grad(std::false_type{});
            tmem_st32(s_buf, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(ds_full);
        }
        const bool dead = nl.x == -INFINITY;  // the row saw no key: its dO gives nothing, whatever it holds
        if (ok && row_ok && hf == 0 && (JOIN && one_tile ? n > 0 : rank == 0)) delta[row_at] = dead ? 0.0f : dl;
        constexpr int HALF = (NB + 1) / 2;
        const int c0 = hf ? HALF : 0, c1 = hf ? NB : HALF;
        const int r0 = sp.q0 + w0;
        const float dq_scale = dead ? 0.0f : args.scale;
        if (!JOIN && ok && rows_ok > 0) {
            if (n == 0) {
                av_store_zero_rows(c0, c1, head * D, r0, dQ, lddq, rows_ok, lane);
            } else if (wait_all(dq_full, 0)) {
                tc_fence_after();
                av_store_rows(tmem_base + lane_addr + 384, dq_scale, c0, c1, sQ + q * (NB * 2048), &tmdQ, head * D, r0,
                              dQ, lddq, rows_ok, lane);
            }
        }
        if constexpr (JOIN) {
            if (ok && n > 0) {
                ok = wait_all(dq_full, 0);
                tc_fence_after();
            }
            // Chunk c (32 columns) is finished by rank c % cluster. The others send it their rows, eight pieces of 16
            // bytes a row, into the rings: [source rank][chunk of the owner][piece][128 queries].
            constexpr int CHUNK = 8 * AV_TILE;
            const int owned = (NB + cluster - 1) / cluster;
            float4* recv = reinterpret_cast<float4*>(sK) + q * 32 + lane;
            const uint32_t acc = tmem_base + lane_addr + 384;
            __syncwarp();
            cluster_sync_all();  // every CTA of the cluster has used its rings
            for (int c = c0; c < c1 && ok && n > 0; ++c) {
                const int owner = c % cluster;
                if (owner == rank) continue;
                uint32_t o[32];
                tmem_ld32(acc + c * 32, o);
                tmem_ld_wait(o);
                const uint32_t to = mapa_shared(smem_u32(recv + (rank * owned + c / cluster) * CHUNK), owner);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    st_cluster_v4(to + k * (AV_TILE * 16), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            __syncwarp();
            cluster_sync_all();
            for (int c = c0; c < c1 && ok && *abort_flag == 0u && rows_ok > 0; ++c) {
                if (c % cluster != rank) continue;
                uint32_t mine[32];
                if (n > 0) {
                    tmem_ld32(acc + c * 32, mine);
                    tmem_ld_wait(mine);
                }
                float sum[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) sum[k] = 0.0f;
                for (int s = 0; s < cluster; ++s) {
                    if (part_begin(s + 1) == part_begin(s) || dq_scale == 0.0f) continue;
                    const float4* from = recv + (s * owned + c / cluster) * CHUNK;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 v = s == rank ? make_float4(__uint_as_float(mine[4 * k]), __uint_as_float(mine[4 * k + 1]),
                                                                 __uint_as_float(mine[4 * k + 2]), __uint_as_float(mine[4 * k + 3]))
                                                   : from[k * AV_TILE];
                        sum[4 * k] += v.x;
                        sum[4 * k + 1] += v.y;
                        sum[4 * k + 2] += v.z;
                        sum[4 * k + 3] += v.w;
                    }
                }
                if (row_ok) {
                    uint4* dst = reinterpret_cast<uint4*>(dQ + static_cast<long long>(r0 + lane) * lddq + head * D + c * 32);
                    const float f = dq_scale;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dst[k] = make_uint4(pack_bf16x2(sum[8 * k] * f, sum[8 * k + 1] * f),
                                            pack_bf16x2(sum[8 * k + 2] * f, sum[8 * k + 3] * f),
                                            pack_bf16x2(sum[8 * k + 4] * f, sum[8 * k + 5] * f),
                                            pack_bf16x2(sum[8 * k + 6] * f, sum[8 * k + 7] * f));
                }
            }
        }
    }
    if (JOIN && warp < 4) av_join_barriers(abort_flag, cluster, warp, lane);

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
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------------------------------
// dK, dV
// ------------------------------------------------------------------------------------------------
template <int D>
struct AvDkvCfg {
    using T = AvTile<D>;
    static constexpr int QST = D == 128 ? 3 : 4;  // a Q tile serves S(i) and, later, dK(i)
    static constexpr int OST = D == 64 ? 4 : D == 96 ? 3 : 2;  // dO: dP(i), then dV(i)
    static constexpr int SST = 2;                 // row statistics
    static constexpr int NUM_BARS = 1 + 2 * QST + 2 * OST + 2 * SST + 8 + 1;
    // 512-byte alignment is what the 64-byte swizzle needs; at D = 128 no more fits
    static constexpr size_t SMEM = 512 + (2 + QST + OST) * size_t(T::BYTES) + SST * 2 * AV_TILE * 4 + 8 * NUM_BARS + 16;
    static_assert(SMEM <= SMEM_LIMIT, "shared memory per block");
    // Columns of tensor memory, all 512 of them: S^T (twice at D = 64), dP^T, dV, dK; P^T over its S^T or, at
    // D = 96, beside it; dS^T over dP^T or, at D = 64, beside P^T in the S^T that both come from
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr int S_BUFS = D == 64 ? 2 : 1;
    static constexpr bool OWN_P = D == 96;
    static constexpr bool BATCH = D <= 96;  // S^T(i+1) does not wait for P^T(i)
    static constexpr uint32_t DP_COL = 128 * S_BUFS;
    static constexpr uint32_t DV_COL = DP_COL + 128;
    static constexpr uint32_t DK_COL = DV_COL + D;
    // columns from one warpgroup's 16-bit values to the other's (64 of each): packed, or in each half of S^T
    static constexpr uint32_t P_COL = OWN_P ? 448 : 0;
    static constexpr uint32_t P_HALF = OWN_P ? 32 : 64;
    static constexpr bool DS_IN_S = S_BUFS == 2;
};

template <int D, bool JOIN>
__global__ void __launch_bounds__(AV_THREADS, 1)
    attn_varlen_dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                           const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
                           const float* LSE, const float* delta, __nv_bfloat16* dK, long long lddk, __nv_bfloat16* dV,
                           long long lddv, int cluster_size, const AvArgs args) {
    const int cluster = JOIN ? cluster_size : 1;
    using Cfg = AvDkvCfg<D>;
    using T = AvTile<D>;
    constexpr int NB = T::NB, QST = Cfg::QST, OST = Cfg::OST, SST = Cfg::SST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 511) & ~uintptr_t(511));
    uint8_t* sK = smem;
    uint8_t* sV = sK + T::BYTES;
    uint8_t* sQ = sV + T::BYTES;
    uint8_t* sdO = sQ + QST * T::BYTES;
    float* stats = reinterpret_cast<float*>(sdO + OST * T::BYTES);  // [SST][-lse2: 128 | -delta: 128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(stats + SST * 2 * AV_TILE);
    uint64_t* kv_full = bars;
    uint64_t* q_full = bars + 1;
    uint64_t* q_empty = q_full + QST;
    uint64_t* do_full = q_empty + QST;
    uint64_t* do_empty = do_full + OST;
    uint64_t* st_full = do_empty + OST;
    uint64_t* st_empty = st_full + SST;
    uint64_t* s_full = st_empty + SST;  // [2]: one per buffer of S^T
    uint64_t* dp_full = s_full + 2;
    uint64_t* p_full = dp_full + 1;
    uint64_t* ds_full = p_full + 1;
    uint64_t* fin_full = ds_full + 1;
    uint64_t* s_read = fin_full + 1;   // one S^T buffer, BATCH: the softmax warps have S^T(i) in registers
    uint64_t* dv_done = s_read + 1;    // OWN_P: P^T(i) has been used
    uint64_t* drain_bar = dv_done + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int item = static_cast<int>(blockIdx.x) / cluster;
    const int rank = JOIN ? static_cast<int>(cluster_ctarank()) : 0;
    const int kvh = item % args.kv_heads;

    grid_dependency_wait();
    AvSpan sp;
    int kt;
    if (!av_pick<AV_TILE, false>(args, item / args.kv_heads, sp, kt)) return;
    const int j0 = kt * AV_TILE;
    const int off = sp.nk - sp.nq;
    // Query tiles start at the first query that sees a key of this tile, not at a multiple of 128: those before it give
    // nothing, and nothing of theirs (a query without keys may hold anything) comes into a product.
    const int qf = args.causal ? max(0, j0 - off) : 0;
    const int rows = max(0, sp.nq - qf), q_row = sp.q0 + qf;
    const int tiles = (rows + AV_TILE - 1) / AV_TILE;
    const int n_all = tiles * args.group;
    // this CTA's part of the iterations
    auto part_begin = [&](int r) { return static_cast<int>(static_cast<long long>(n_all) * r / cluster); };
    const int it0 = part_begin(rank);
    const int n = part_begin(rank + 1) - it0;
    const int q_tail = tiles * AV_TILE > rows ? rows - (tiles - 1) * AV_TILE : AV_TILE;
    // Iterations: the group's heads in turn, of each the query tiles. Every role walks them
    // with counters (a division an iteration was a tenth of the loop).
    struct Walk {
        int head, tile, tiles;
        __device__ __forceinline__ void next() {
            if (++tile == tiles) {
                tile = 0;
                ++head;
            }
        }
    };
    const Walk first{kvh * args.group + (n > 0 ? it0 / tiles : 0), n > 0 ? it0 % tiles : 0, tiles};

    // Row statistics of a query tile, four rows a lane of warp 2; the first are asked for before the set-up.
    constexpr int ST_ROWS = AV_TILE / 32;
    float st_lse[ST_ROWS], st_delta[ST_ROWS];
    Walk st_walk = first;
    auto st_fetch = [&]() {
        const int i0 = st_walk.tile * AV_TILE + lane;
        const long long at = static_cast<long long>(st_walk.head) * args.Tq + q_row + i0;
#pragma unroll
        for (int r = 0; r < ST_ROWS; ++r) {
            const bool row_ok = i0 + r * 32 < rows;
            st_lse[r] = row_ok ? LSE[at + r * 32] : -INFINITY;
            st_delta[r] = row_ok ? delta[at + r * 32] : 0.0f;
        }
    };
    if (warp == 2 && n > 0) st_fetch();

    if (threadIdx.x == 0) {
        mbar_init(kv_full, 2);
        for (int i = 0; i < QST; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < OST; ++i) {
            mbar_init(&do_full[i], 1);
            mbar_init(&do_empty[i], 1);
        }
        for (int i = 0; i < SST; ++i) {
            mbar_init(&st_full[i], 1);
            mbar_init(&st_empty[i], 8);
        }
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(dp_full, 1);
        mbar_init(p_full, 8);
        mbar_init(ds_full, 8);
        mbar_init(fin_full, 1);
        mbar_init(s_read, 8);
        mbar_init(dv_done, 1);
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        if (n > 0 && !av_starved(args, rank, cluster)) {
            av_load<D>(sK, &tmK, kv_full, kvh, sp.k0 + j0);
            av_load<D>(sQ, &tmQ, &q_full[0], first.head, q_row + first.tile * AV_TILE);
            av_load<D>(sV, &tmV, kv_full, kvh, sp.k0 + j0);
            av_load<D>(sdO, &tmdO, &do_full[0], first.head, q_row + first.tile * AV_TILE);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_launch_dependents();  // once this CTA holds its tensor memory: a dependent may want some too
    const Ctl ctl{args.status, abort_flag, args.budget_ns};
    auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool got = wait_bounded(bar, parity, ctl);
        return __all_sync(0xffffffffu, got) != 0;
    };

    if (warp < 4) {
        reg_dealloc<T::REGS_CTRL>();
        if (warp == 0) {
            if (lane == 0) {
                // ---------------- TMA producer ----------------
                bool ok = true;
                Walk w = first;
                for (int it = 1; it < n && ok; ++it) {
                    w.next();
                    int st = it % QST;
                    ok = wait_bounded(&q_empty[st], ((it / QST) & 1) ^ 1u, ctl);
                    if (!ok) break;
                    av_load<D>(sQ + st * T::BYTES, &tmQ, &q_full[st], w.head, q_row + w.tile * AV_TILE);
                    st = it % OST;
                    ok = wait_bounded(&do_empty[st], ((it / OST) & 1) ^ 1u, ctl);
                    if (!ok) break;
                    av_load<D>(sdO + st * T::BYTES, &tmdO, &do_full[st], w.head, q_row + w.tile * AV_TILE);
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            constexpr uint32_t IDESC_S = make_idesc_bf16(AV_TILE, AV_TILE, false, false);
            constexpr uint32_t IDESC_G = make_idesc_bf16(AV_TILE, D, false, true);
            const uint64_t k_desc = make_sdesc_sw64(smem_u32(sK), 16, 512);
            const uint64_t v_desc = make_sdesc_sw64(smem_u32(sV), 16, 512);
            const uint64_t q_desc = make_sdesc_sw64(smem_u32(sQ), 16, 512);
            const uint64_t qt_desc = make_sdesc_sw64(smem_u32(sQ), T::BOX, 512);  // queries summed over
            const uint64_t do_desc = make_sdesc_sw64(smem_u32(sdO), 16, 512);
            const uint64_t dot_desc = make_sdesc_sw64(smem_u32(sdO), T::BOX, 512);
            auto score = [&](uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t o = ((k >> 1) * T::BOX + (k & 1) * 32) >> 4;
                    umma_bf16_elect(d, a + o, b + o, IDESC_S, k > 0 ? 1u : 0u);
                }
            };
            auto grad = [&](uint32_t d, uint32_t a, uint32_t half, uint64_t b, bool fresh) {
#pragma unroll
                for (int k = 0; k < AV_TILE / 16; ++k)
                    umma_bf16_ts_elect(d, a + (k >> 2) * half + (k & 3) * 8, b + ((k * 1024) >> 4), IDESC_G,
                                       k > 0 || !fresh ? 1u : 0u);
            };
            AvRing<QST> q_ahead, q_sum;            // Q tiles of the next S^T and of the next dK
            AvRing<OST> do_ahead, do_dp, do_sum;   // dO tiles waited for, of the next dP^T and of the next dV
            auto off = [&](int st) { return static_cast<uint32_t>((st * T::BYTES) >> 4); };
            Walk ahead = first;  // the iteration whose tiles have been waited for
            auto tiles_wait = [&]() {
                if (!wait_all(&q_full[q_ahead.st], q_ahead.ph) || !wait_all(&do_full[do_ahead.st], do_ahead.ph)) return false;
                if (q_tail < AV_TILE && ahead.tile == tiles - 1) {
                    av_clear_rows<D>(sQ + q_ahead.st * T::BYTES, q_tail, lane);
                    av_clear_rows<D>(sdO + do_ahead.st * T::BYTES, q_tail, lane);
                }
                do_ahead.next();
                return true;
            };
            auto s_buf = [&](int it) { return Cfg::S_BUFS == 2 ? (it & 1) : 0; };
            auto s_mma = [&](int it) {
                score(tmem_base + s_buf(it) * 128, k_desc, q_desc + off(q_ahead.st));
                umma_commit_elect(&s_full[s_buf(it)]);
                q_ahead.next();
            };
            auto dp_mma = [&]() {
                score(tmem_base + Cfg::DP_COL, v_desc, do_desc + off(do_dp.st));
                umma_commit_elect(dp_full);
                do_dp.next();
            };
            auto dv_mma = [&](int it) {  // dV += P^T dO
                grad(tmem_base + Cfg::DV_COL, tmem_base + (Cfg::OWN_P ? Cfg::P_COL : s_buf(it) * 128), Cfg::P_HALF,
                     dot_desc + off(do_sum.st), it == 0);
                umma_commit_elect(&do_empty[do_sum.st]);
                do_sum.next();
                if (Cfg::OWN_P) umma_commit_elect(dv_done);
            };
            auto dk_mma = [&](int it) {  // dK += dS^T Q
                grad(tmem_base + Cfg::DK_COL, tmem_base + (Cfg::DS_IN_S ? s_buf(it) * 128 + 32 : Cfg::DP_COL), 64,
                     qt_desc + off(q_sum.st), it == 0);
                umma_commit_elect(&q_empty[q_sum.st]);
                q_sum.next();
            };
            bool ok = n > 0 && wait_all(kv_full, 0) && tiles_wait();
            if (ok) {
                tc_fence_after();
                s_mma(0);
                dp_mma();
            }
            if constexpr (Cfg::BATCH) {
                // One wait on the softmax an iteration, and all its products behind it, dP^T (which the softmax
                // needs next) as soon as its columns are free; S^T runs two iterations ahead.
                auto s_ahead = [&](int it) -> bool {  // S^T(it): over P^T(it-2), or once S^T(it-1) has been read
                    ahead.next();
                    if (!tiles_wait() || (Cfg::S_BUFS == 1 && !wait_all(s_read, (it - 1) & 1))) return false;
                    tc_fence_after();
                    s_mma(it);
                    return true;
                };
                if (ok && n > 1) ok = s_ahead(1);
                for (int it = 0; it < n && ok; ++it) {
                    if (!(ok = wait_all(ds_full, it & 1))) break;
                    tc_fence_after();
                    if (!Cfg::DS_IN_S) dk_mma(it);
                    if (it + 1 < n) dp_mma();
                    dv_mma(it);
                    if (Cfg::DS_IN_S) dk_mma(it);
                    if (it + 2 < n) ok = s_ahead(it + 2);
                }
            } else {
                for (int it = 0; it < n && ok; ++it) {
                    // The next tiles are waited for (and a tail cleared) before this iteration's softmax is, so
                    // that nothing lies between the products that follow it.
                    const bool more = it + 1 < n;
                    if (more) {
                        ahead.next();
                        if (!(ok = tiles_wait())) break;
                    }
                    if (!(ok = wait_all(p_full, it & 1))) break;
                    tc_fence_after();
                    dv_mma(it);
                    if (more) s_mma(it + 1);  // over P^T(i), whose product was issued before it
                    if (!(ok = wait_all(ds_full, it & 1))) break;
                    tc_fence_after();
                    dk_mma(it);
                    if (more) dp_mma();
                }
            }
            if (ok) umma_commit_elect(fin_full);
            umma_commit_elect(drain_bar);
            wait_drain(drain_bar, 0, args.status);
        } else if (warp == 2) {
            // ---------------- row statistics of each query tile ----------------
            // One iteration's values are in registers before the buffer of the one before last is free.
            for (int it = 0; it < n; ++it) {
                const int st = it % SST;
                if (!wait_all(&st_empty[st], ((it / SST) & 1) ^ 1u)) break;
                float* s = stats + st * 2 * AV_TILE + lane;
#pragma unroll
                for (int r = 0; r < ST_ROWS; ++r) {
                    s[r * 32] = -lse_to_log2(st_lse[r]);
                    s[AV_TILE + r * 32] = -st_delta[r];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&st_full[st]);
                st_walk.next();
                if (it + 1 < n) st_fetch();
            }
        }
    } else {
        reg_alloc<T::REGS_SOFTMAX>();
        // ---------------- softmax: warps 4..7 query columns 0..63, warps 8..11 columns 64..127 ----------------
        // The scores are read as matrix fragments, four keys of a thread with 16 columns each, rather than one
        // key with 64: the statistics go by column, and a thread then fetches 16 of each from shared memory
        // instead of 64 (with 64, those loads took 1290 of an iteration's cycles on the load pipe).
        const int hf = (warp - 4) >> 2;
        const int q = warp & 3;
        const int w0 = j0 + q * 32;   // first key of this warp, in its sequence
        const int rows_ok = min(32, sp.nk - w0);
        const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t dp_addr = tmem_base + lane_addr + Cfg::DP_COL + hf * 64;
        const float2 c2v = make_float2(args.scale_log2, args.scale_log2);
        Walk at = first;
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int st = it % SST;
            // this thread's columns 8 i + 2 (lane % 4), + 1 of its warps' half of the tile
            const float2* nl = reinterpret_cast<const float2*>(stats + st * 2 * AV_TILE + hf * 64) + (lane & 3);
            const float2* nd = nl + AV_TILE / 2;
            const int sb = Cfg::S_BUFS == 2 ? (it & 1) : 0;
            const uint32_t s_addr = tmem_base + lane_addr + sb * 128 + hf * 64;
            const uint32_t p_addr = Cfg::OWN_P ? tmem_base + lane_addr + Cfg::P_COL + hf * Cfg::P_HALF : s_addr;
            const uint32_t ds_addr = Cfg::DS_IN_S ? s_addr + 32 : dp_addr;
            if (!(ok = wait_all(&st_full[st], (it / SST) & 1) &&
                       wait_all(&s_full[sb], (Cfg::S_BUFS == 2 ? it >> 1 : it) & 1)))
                break;
            tc_fence_after();
            // 32 keys x 64 queries of the warp as two fragments of 16 keys: keys f * 16 + e * 8 + lane / 4
            uint32_t p[2][32], w[2][16];
            tmem_ld_frag64(s_addr, p[0]);
            tmem_ld_frag64(s_addr + (16u << 16), p[1]);
            float2 row[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) row[i] = nl[i * 4];
            tmem_wait_ld();
            reg_fence32(p[0]);
            reg_fence32(p[1]);
            if (Cfg::BATCH && Cfg::S_BUFS == 1) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read);
            }
            // causal: a key is visible from column lo on; lo_w, the most, is the warp's last key's
            const int lo_w = args.causal ? w0 + 31 - off - qf - at.tile * AV_TILE - hf * 64 : 0;
            const int lo = lo_w - 31 + (lane >> 2) - 2 * (lane & 3);  // of key lane / 4, against column 8 i + c
            auto prob = [&](auto masked) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int fe = 0; fe < 4; ++fe) {
                        const int f = fe >> 1, e = fe & 1;
                        uint32_t& a = p[f][4 * i + 2 * e];
                        uint32_t& b = p[f][4 * i + 2 * e + 1];
                        const float2 x = fma2(make_float2(__uint_as_float(a), __uint_as_float(b)), c2v, row[i]);
                        float2 pr = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        if (decltype(masked)::value) {
                            pr.x = 8 * i >= lo + f * 16 + e * 8 ? pr.x : 0.0f;
                            pr.y = 8 * i + 1 >= lo + f * 16 + e * 8 ? pr.y : 0.0f;
                        }
                        a = __float_as_uint(pr.x);
                        b = __float_as_uint(pr.y);
                        w[f][2 * i + e] = pack_bf16x2(pr.x, pr.y);
                    }
            };
            if (args.causal && lo_w > 0)
                prob(std::true_type{});
            else
                prob(std::false_type{});
            if (Cfg::OWN_P && it > 0 && !(ok = wait_all(dv_done, (it - 1) & 1))) break;
            tmem_st_frag32(p_addr, w[0]);
            tmem_st_frag32(p_addr + (16u << 16), w[1]);
            if (!Cfg::BATCH) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) row[i] = nd[i * 4];
            if (!(ok = wait_all(dp_full, it & 1))) break;
            tc_fence_after();
            uint32_t t[2][32];
            tmem_ld_frag64(dp_addr, t[0]);
            tmem_ld_frag64(dp_addr + (16u << 16), t[1]);
            tmem_wait_ld();
            reg_fence32(t[0]);
            reg_fence32(t[1]);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int fe = 0; fe < 4; ++fe) {
                    const int f = fe >> 1, e = fe & 1, k = 4 * i + 2 * e;
                    const float2 dp = make_float2(__uint_as_float(t[f][k]), __uint_as_float(t[f][k + 1]));
                    const float2 pr = make_float2(__uint_as_float(p[f][k]), __uint_as_float(p[f][k + 1]));
                    const float2 ds = mul2(pr, add2(dp, row[i]));
                    w[f][2 * i + e] = pack_bf16x2(ds.x, ds.y);
                }
            tmem_st_frag32(ds_addr, w[0]);
            tmem_st_frag32(ds_addr + (16u << 16), w[1]);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&st_empty[st]);
                mbar_arrive(ds_full);
            }
            at.next();
        }
        __nv_bfloat16* out = hf ? dK : dV;
        const long long ld = hf ? lddk : lddv;
        if (!JOIN && ok && rows_ok > 0) {
            // warps 4..7 write dV, warps 8..11 dK; K's and V's tiles are free for the staging
            if (n == 0) {
                av_store_zero_rows(0, NB, kvh * D, sp.k0 + w0, out, ld, rows_ok, lane);
            } else if (wait_all(fin_full, 0)) {
                tc_fence_after();
                av_store_rows(tmem_base + lane_addr + (hf ? Cfg::DK_COL : Cfg::DV_COL), hf ? args.scale : 1.0f, 0, NB,
                              (hf ? sK : sV) + q * (NB * 2048), hf ? &tmdK : &tmdV, kvh * D, sp.k0 + w0, out, ld,
                              rows_ok, lane);
            }
        }
        if constexpr (JOIN) {
            if (ok && n > 0) {
                ok = wait_all(fin_full, 0);
                tc_fence_after();
            }
            // Chunk c (32 columns) of dV or dK is finished by rank (hf NB + c) % cluster. The others send it
            // their rows, eight pieces of 16 bytes a row, into the ring of Q and dO tiles:
            // [source rank][chunk of the owner][piece][128 keys].
            constexpr int CHUNK = 8 * AV_TILE;
            const int owned = (2 * NB + cluster - 1) / cluster;
            float4* recv = reinterpret_cast<float4*>(sQ);
            const uint32_t acc = tmem_base + lane_addr + (hf ? Cfg::DK_COL : Cfg::DV_COL);
            __syncwarp();
            cluster_sync_all();  // every CTA of the cluster has used its ring
            for (int c = 0; c < NB && ok && n > 0; ++c) {
                const int id = hf * NB + c, owner = id % cluster;
                if (owner == rank) continue;
                uint32_t o[32];
                tmem_ld32(acc + c * 32, o);
                tmem_ld_wait(o);
                const uint32_t to = mapa_shared(
                    smem_u32(recv + (rank * owned + id / cluster) * CHUNK + q * 32 + lane), owner);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    st_cluster_v4(to + k * (AV_TILE * 16), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            __syncwarp();
            cluster_sync_all();
            const float f = hf ? args.scale : 1.0f;
            for (int c = 0; c < NB && ok && *abort_flag == 0u; ++c) {
                const int id = hf * NB + c;
                if (id % cluster != rank) continue;
                uint32_t mine[32];
                if (n > 0) {
                    tmem_ld32(acc + c * 32, mine);
                    tmem_ld_wait(mine);
                }
                float sum[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) sum[k] = 0.0f;
                for (int r = 0; r < cluster; ++r) {
                    if (part_begin(r + 1) == part_begin(r)) continue;  // a rank without a part has no sums
                    const float4* from = recv + (r * owned + id / cluster) * CHUNK + q * 32 + lane;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 v = r == rank ? make_float4(__uint_as_float(mine[4 * k]), __uint_as_float(mine[4 * k + 1]),
                                                                 __uint_as_float(mine[4 * k + 2]), __uint_as_float(mine[4 * k + 3]))
                                                   : from[k * AV_TILE];
                        sum[4 * k] += v.x;
                        sum[4 * k + 1] += v.y;
                        sum[4 * k + 2] += v.z;
                        sum[4 * k + 3] += v.w;
                    }
                }
                if (lane < rows_ok) {
                    uint4* dst = reinterpret_cast<uint4*>(out + static_cast<long long>(sp.k0 + w0 + lane) * ld + kvh * D + c * 32);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dst[k] = make_uint4(pack_bf16x2(sum[8 * k] * f, sum[8 * k + 1] * f),
                                            pack_bf16x2(sum[8 * k + 2] * f, sum[8 * k + 3] * f),
                                            pack_bf16x2(sum[8 * k + 4] * f, sum[8 * k + 5] * f),
                                            pack_bf16x2(sum[8 * k + 6] * f, sum[8 * k + 7] * f));
                }
            }
        }
    }
    if (JOIN && warp < 4) av_join_barriers(abort_flag, cluster, warp, lane);

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
        tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
    }
}

// CTAs that share a key tile. The estimate, in iterations (a head's query tile each): the larger of the longest
// CTA and of all the work over the SMs that clusters of this size can use, where each CTA costs three
// iterations more than its own, and one of a cluster seven to ten (its set-up, the join, and SMs that wait for
// the cluster's others). Lengths are on the device: the sum over the sequences is taken between that of equal
// ones and that of the longest. Measured with 1, 2, 4, 8 CTAs a tile: 16,384 causal queries, eight heads on two,
// d = 128 (256 tiles, the longest 512 iterations) 782, 727, 785, 1083 us; eight packed documents, 16 heads on
// four, d = 96 (272 tiles, the longest 76) 109, 112, 161, 335 us.
static int dkv_cluster(const AvArgs& a, int sms) {
    const double tiles = a.Tk / double(AV_TILE) + 0.5 * a.nseq;
    const double longest = double(a.group) * ceil_div(a.max_q, AV_TILE);
    const double mean = double(a.Tq) / a.nseq;
    const double total = tiles * a.heads * (0.5 * (a.max_q + mean) / AV_TILE + 0.5) * (a.causal ? 0.5 : 1.0);
    const double extra[4] = {3.0, 7.0, 8.0, 10.0};
    return av_cluster(tiles * a.kv_heads, longest, total, extra, 4, sms);
}

// CTAs that share a query tile, as the key kernel below shares key tiles; iterations are key tiles. A CTA costs five more
// than its own, one of a cluster nine to fourteen. Measured with 1, 2, 4, 8, both kernels: one query on 16,384 keys, eight
// heads, d = 128, the same tensors every time, 157, 100, 71, 60 us (88 where they come from memory); 4096 causal queries, d = 64, one head 44, 34, 29, 40, eight heads 64, 80, 106, 180.
static int dq_cluster(const AvArgs& a, int sms) {
    const double items = double(av_max_tiles(a.nseq, a.Tq, a.max_q, AV_TILE)) * a.heads;
    const double extra[4] = {5.0, 9.0, 12.0, 14.0};
    return av_cluster(items, ceil_div(a.max_k, AV_TILE), items * av_mean_keys(a), extra, 2, sms);
}

struct AvBwdMaps {
    CUtensorMap q, k, v, d_o, dq, dk, dv;
};

template <int D>
static cudaError_t launch_bwd(const AvBwdMaps& m, const mp_bf16* O, long long ldo, const mp_bf16* dO, long long lddo,
                              const float* LSE, float* delta, mp_bf16* dQ, long long lddq, mp_bf16* dK, long long lddk,
                              mp_bf16* dV, long long lddv, const AvArgs& a, int sms, cudaStream_t s) {
    auto bf = [](auto* p) { return reinterpret_cast<__nv_bfloat16*>(const_cast<mp_bf16*>(p)); };
    const long long qtiles = av_max_tiles(a.nseq, a.Tq, a.max_q, AV_TILE), ktiles = av_max_tiles(a.nseq, a.Tk, a.max_k, AV_TILE);
    cudaError_t e = cudaSuccess;
    if (qtiles > 0) {
        const int cluster = dq_cluster(a, sms);
        auto kern = cluster > 1 ? attn_varlen_dq_kernel<D, true> : attn_varlen_dq_kernel<D, false>;
        e = av_launch(kern, qtiles * a.heads * cluster, cluster, AvDqCfg<D>::SMEM, s, m.q, m.k, m.v, m.d_o, m.dq,
                      static_cast<const __nv_bfloat16*>(bf(O)), ldo, static_cast<const __nv_bfloat16*>(bf(dO)), lddo, LSE, delta,
                      bf(dQ), lddq, cluster, a);
    }
    if (e == cudaSuccess && ktiles > 0) {
        const int cluster = dkv_cluster(a, sms);
        auto kern = cluster > 1 ? attn_varlen_dkv_kernel<D, true> : attn_varlen_dkv_kernel<D, false>;
        e = av_launch(kern, ktiles * a.kv_heads * cluster, cluster, AvDkvCfg<D>::SMEM, s,
                      m.q, m.k, m.v, m.d_o, m.dk, m.dv, LSE, static_cast<const float*>(delta), bf(dK), lddk, bf(dV),
                      lddv, cluster, a);
    }
    return e;
}

}  // namespace mptp

using namespace mptp;

extern "C" mp_status mp_attn_varlen_bwd(const mp_bf16* Q, const mp_bf16* K, const mp_bf16* V, const mp_bf16* O,
                                        const float* LSE, const mp_bf16* dO, mp_bf16* dQ, mp_bf16* dK, mp_bf16* dV,
                                        float* delta_ws, const int32_t* cu_q, const int32_t* cu_k, int nseq, int Tq,
                                        int Tk, int max_q, int max_k, int heads, int kv_heads, int d, long long ldq,
                                        long long ldk, long long ldv, long long ldo, long long lddo, long long lddq,
                                        long long lddk, long long lddv, int causal, float scale, uint32_t* d_status,
                                        void* stream) {
    mp_status st = av_check(nseq, Tq, Tk, max_q, max_k, heads, kv_heads, d, scale);
    if (st != MP_OK) return st;
    const long long qw = static_cast<long long>(heads) * d, kw = static_cast<long long>(kv_heads) * d;
    if (av_bad_pitch(ldq, qw) || av_bad_pitch(ldo, qw) || av_bad_pitch(lddo, qw) || av_bad_pitch(lddq, qw) ||
        av_bad_pitch(ldk, kw) || av_bad_pitch(ldv, kw) || av_bad_pitch(lddk, kw) || av_bad_pitch(lddv, kw))
        return MP_ERR_UNSUPPORTED_SHAPE;
    if (nseq == 0 || (max_q == 0 && max_k == 0)) return MP_OK;
    if (!cu_q || !cu_k || (Tq > 0 && (!Q || !O || !LSE || !dO || !dQ || !delta_ws)) || (Tk > 0 && (!K || !V || !dK || !dV)))
        return MP_ERR_INVALID_ARG;
    const void* ptrs[] = {Q, K, V, O, dO, dQ, dK, dV};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MP_ERR_MISALIGNED;
    const void* words[] = {LSE, delta_ws, cu_q, cu_k, d_status};
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return MP_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_device(&sms)) != MP_OK) return st;

    // A side without rows is never loaded or stored: its maps take the other side's tensors.
    const int qc = static_cast<int>(qw), kc = static_cast<int>(kw);
    AvBwdMaps m{};
    bool ok = true;
    if (Tq > 0)
        ok = av_tmap(&m.q, Q, qc, Tq, ldq, d) && av_tmap(&m.d_o, dO, qc, Tq, lddo, d) && make_tmap_bf16_out(&m.dq, dQ, qc, Tq, lddq);
    if (ok && Tk > 0)
        ok = av_tmap(&m.k, K, kc, Tk, ldk, d) && av_tmap(&m.v, V, kc, Tk, ldv, d) && make_tmap_bf16_out(&m.dk, dK, kc, Tk, lddk) &&
             make_tmap_bf16_out(&m.dv, dV, kc, Tk, lddv);
    if (!ok) return MP_ERR_CUDA;
    if (Tq == 0) m.q = m.d_o = m.dq = m.k;
    if (Tk == 0) m.k = m.v = m.dk = m.dv = m.q;
    const AvArgs a = av_args(cu_q, cu_k, nseq, Tq, Tk, max_q, max_k, heads, kv_heads, causal ? 1 : 0, scale, d_status);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        d == 64   ? launch_bwd<64>(m, O, ldo, dO, lddo, LSE, delta_ws, dQ, lddq, dK, lddk, dV, lddv, a, sms, s)
        : d == 96 ? launch_bwd<96>(m, O, ldo, dO, lddo, LSE, delta_ws, dQ, lddq, dK, lddk, dV, lddv, a, sms, s)
                  : launch_bwd<128>(m, O, ldo, dO, lddo, LSE, delta_ws, dQ, lddq, dK, lddk, dV, lddv, a, sms, s);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
