// Entry point of the packed attention's forward: mp_attn_varlen_fwd.
//
//   S = scale Q K^T (+ causal mask),  LSE = log sum_k exp S,  O = exp(S - LSE) V
// over packed sequences of any lengths, key heads shared by groups of query heads.
//
// One CTA per (sequence, query head, pair of consecutive 128-query tiles), 384 threads, as the
// attention block's kernel (mptp_attn.cu) with its whole sequences of 128-row tiles: the two query
// tiles A and B share every key and value tile, so each is loaded once for 256 queries.
//   warp 0: TMA producer (both query tiles, then rings of K and V tiles)
//   warp 1: TMEM and the products: per key tile j and query tile g, O_g += P_g V_j (P_g from TMEM), then
//           S_g(j+1) = Q_g K_{j+1}^T over the same columns; the tensor core works on one query tile
//           while the other's softmax runs. It also clears the rows of the last value tile that belong
//           to the next sequence.
//   warpgroups 1, 2: softmax of tile A and of tile B, thread = query row. Running maximum, raised (and O
//           and the sum rescaled) only when it grows by more than 2^8; the sum is kept in fp32 over the
//           unrounded probabilities, which are rounded to bf16 for the product with V.
// Bound by the hand-overs between softmax and products, not by either's rate: a pair of key tiles takes 2800 to 3060
// cycles, in which the tensor core has 1024 (D = 64) to 2048 (D = 128) of work and the exponentials 1024. 4096 tokens,
// 19 heads, not causal: 93, 101 and 113 us for D = 64, 96, 128 (0.88, 1.22, 1.44 PFLOP/s). At D = 64, P in columns of
// its own, so that the next scores are computed beside the softmax, made this kernel 5 % faster and a training step no
// faster; the two tiles taking turns at the exponentials made it 9 % slower.
// Where few query tiles have long rows of keys, a cluster of two to eight CTAs shares a pair of query tiles: each takes a
// part of its key tiles, and maxima, sums and fp32 outputs are joined through distributed shared memory in rank order.
// Masked scores are replaced, not added to, and other sequences' rows of V are cleared, so that no value of theirs
// reaches a row. A hidden key of the row's own sequence has the weight 0 in the product with V: an infinity or NaN in
// its V makes O of the rows of its tile NaN, as the definition's product does. A row without keys gets O = 0 and
// LSE = -inf whatever its tile holds.
#include <type_traits>

#include "mptp_attn_varlen.cuh"

namespace mptp {

constexpr float AV_RESCALE_LOG2 = 8.0f;  // lazy rescale threshold on the maximum, exp2 domain

template <int D>
struct AvFwdCfg {
    using T = AvTile<D>;
    // D = 128: two query tiles and five key or value tiles of 32 KB fill the shared memory
    static constexpr int KST = D == 64 ? 4 : 3;
    static constexpr int VST = D == 64 ? 4 : D == 96 ? 3 : 2;
    static constexpr int NUM_BARS = 2 + 2 * KST + 2 * VST + 2 * 3 + 1;
    static constexpr size_t SMEM = 1024 + (2 + KST + VST) * size_t(T::BYTES) + 8 * NUM_BARS + 16;
    static_assert(SMEM <= SMEM_LIMIT, "shared memory per block");
    static_assert((KST + VST) * T::BYTES >= 8 * AV_TILE * 128, "a chunk of every part at the join");
    static constexpr uint32_t TMEM_COLS = 512;  // S_A, S_B at 0, 128; O_A, O_B at 256, 384
};

template <int D, bool JOIN>
__global__ void __launch_bounds__(AV_THREADS, 1)
    attn_varlen_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                           __nv_bfloat16* O, long long ldo, float* LSE, int cluster_size, const AvArgs args) {
    const int cluster = JOIN ? cluster_size : 1;
    using Cfg = AvFwdCfg<D>;
    using T = AvTile<D>;
    constexpr int NB = T::NB, KST = Cfg::KST, VST = Cfg::VST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;                     // tile g at g * BYTES
    uint8_t* sK = sQ + 2 * T::BYTES;
    uint8_t* sV = sK + KST * T::BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sV + VST * T::BYTES);
    uint64_t* q_full = bars;                // [2]
    uint64_t* k_full = bars + 2;
    uint64_t* k_empty = k_full + KST;
    uint64_t* v_full = k_empty + KST;
    uint64_t* v_empty = v_full + VST;
    uint64_t* s_full = v_empty + VST;       // [2]: S_g computed (and every earlier product of tile g)
    uint64_t* p_full = s_full + 2;          // [2]: P_g in TMEM (and O_g rescaled)
    uint64_t* o_full = p_full + 2;          // [2]: last P_g V done
    uint64_t* drain_bar = o_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
    volatile uint32_t* abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int item = static_cast<int>(blockIdx.x) / cluster;
    const int rank = JOIN ? static_cast<int>(cluster_ctarank()) : 0;
    const int head = item % args.heads;  // heads of one sequence side by side
    const int kvh = head / args.group;

    grid_dependency_wait();  // the sequences' offsets, like the tensors, may come from the kernel before
    AvSpan sp;
    int pr;
    if (!av_pick<2 * AV_TILE, true>(args, item / args.heads, sp, pr))
        return;
    const int qt[2] = {2 * pr, 2 * pr + 1};
    int nt[2] = {av_key_tiles(sp, qt[0] * AV_TILE, args.causal), av_key_tiles(sp, qt[1] * AV_TILE, args.causal)};
    int n = max(nt[0], nt[1]);
    int kb = 0;  // first key of this CTA's part, in the sequence
    if constexpr (JOIN) {
        const int b0 = n * rank / cluster, b1 = n * (rank + 1) / cluster;
        for (int g = 0; g < 2; ++g) nt[g] = max(0, min(nt[g], b1) - b0);
        n = max(nt[0], nt[1]);
        kb = b0 * AV_TILE;
    }
    const int k_row = sp.k0 + kb;
    const int v_tail = n * AV_TILE > sp.nk - kb ? sp.nk - kb - (n - 1) * AV_TILE : AV_TILE;  // own rows of the last tile

    if (threadIdx.x == 0) {
        for (int g = 0; g < 2; ++g) {
            mbar_init(&q_full[g], 1);
            mbar_init(&s_full[g], 1);
            mbar_init(&p_full[g], 4);
            mbar_init(&o_full[g], 1);
        }
        for (int i = 0; i < KST; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < VST; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0u;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        // The first loads overlap the rest of the set-up.
        const bool starved = av_starved(args, rank, cluster);
        if (n > 0 && !starved) av_load<D>(sK, &tmK, &k_full[0], kvh, k_row);
        for (int g = 0; g < 2; ++g)
            if (nt[g] > 0 && !starved) av_load<D>(sQ + g * T::BYTES, &tmQ, &q_full[g], head, sp.q0 + qt[g] * AV_TILE);
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
                constexpr int LEAD = KST - 1;  // K tiles loaded ahead of the V tile of the same index
                auto load = [&](int j, const CUtensorMap* map, uint64_t* full, uint64_t* empty, uint8_t* ring,
                                int stages) -> bool {
                    const int st = j % stages;
                    if (!wait_bounded(&empty[st], ((j / stages) & 1) ^ 1u, ctl)) return false;
                    av_load<D>(ring + st * T::BYTES, map, &full[st], kvh, k_row + j * AV_TILE);
                    return true;
                };
                bool ok = true;
                for (int j = 1; j < LEAD && j < n && ok; ++j) ok = load(j, &tmK, k_full, k_empty, sK, KST);
                for (int j = 0; j < n && ok; ++j) {
                    if (j + LEAD < n) ok = load(j + LEAD, &tmK, k_full, k_empty, sK, KST);
                    if (ok) ok = load(j, &tmV, v_full, v_empty, sV, VST);
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issuer (whole warp, one elected lane issues) ----------------
            constexpr uint32_t IDESC_S = make_idesc_bf16(AV_TILE, AV_TILE, false, false);
            constexpr uint32_t IDESC_PV = make_idesc_bf16(AV_TILE, D, false, true);
            const uint64_t q_desc = make_sdesc_sw64(smem_u32(sQ), 16, 512);
            const uint64_t k_desc = make_sdesc_sw64(smem_u32(sK), 16, 512);
            const uint64_t v_desc = make_sdesc_sw64(smem_u32(sV), T::BOX, 512);
            auto s_mma = [&](int g, int j) {
                const uint64_t qd = q_desc + static_cast<uint32_t>((g * T::BYTES) >> 4);
                const uint64_t kd = k_desc + static_cast<uint32_t>(((j % KST) * T::BYTES) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 1) * T::BOX + (k & 1) * 32) >> 4;
                    umma_bf16_elect(tmem_base + g * 128, qd + off, kd + off, IDESC_S, k > 0 ? 1u : 0u);
                }
                umma_commit_elect(&s_full[g]);
            };
            auto pv_mma = [&](int g, int j) {
                const uint64_t vd = v_desc + static_cast<uint32_t>(((j % VST) * T::BYTES) >> 4);
                const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
                for (int k = 0; k < AV_TILE / 16; ++k)
                    umma_bf16_ts_elect(tmem_base + 256 + g * 128, tmem_base + g * 128 + k * 8, vd + ((k * 1024) >> 4),
                                       IDESC_PV, k > 0 ? 1u : acc0);
            };
            bool ok = n == 0 || wait_all(&k_full[0], 0);
            for (int g = 0; g < 2 && ok && n > 0; ++g) {
                if (nt[g] == 0) continue;
                ok = wait_all(&q_full[g], 0);
                if (!ok) break;
                tc_fence_after();
                s_mma(g, 0);
            }
            if (ok && n > 0) umma_commit_elect(&k_empty[0]);
            for (int j = 0; j < n && ok; ++j) {
                ok = wait_all(&v_full[j % VST], (j / VST) & 1);
                if (ok && j == n - 1 && v_tail < AV_TILE) av_clear_rows<D>(sV + (j % VST) * T::BYTES, v_tail, lane);
                bool k_next = false;  // K tile j + 1 waited for
                for (int g = 0; g < 2 && ok; ++g) {
                    if (j >= nt[g]) continue;
                    if (!wait_all(&p_full[g], j & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    pv_mma(g, j);
                    if (j + 1 < nt[g]) {
                        if (!k_next) {
                            if (!wait_all(&k_full[(j + 1) % KST], ((j + 1) / KST) & 1)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            k_next = true;
                        }
                        s_mma(g, j + 1);
                    } else {
                        umma_commit_elect(&o_full[g]);
                    }
                }
                if (!ok) break;
                umma_commit_elect(&v_empty[j % VST]);
                if (k_next) umma_commit_elect(&k_empty[(j + 1) % KST]);
            }
            umma_commit_elect(drain_bar);  // every MMA must finish before TMEM is freed
            wait_drain(drain_bar, 0, args.status);
        }
    } else {
        reg_alloc<T::REGS_SOFTMAX>();
        // ---------------- softmax (warps 4..7: tile A, 8..11: tile B) ----------------
        const int g = (warp - 4) >> 2;
        const int q = warp & 3;                               // TMEM lane quarter
        const int w0 = qt[g] * AV_TILE + q * 32;              // first query of this warp, in its sequence
        const int qi = w0 + lane;
        const int ng = nt[g];
        const int rows_ok = min(32, sp.nq - w0);              // <= 0: no rows
        const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t s_addr = tmem_base + lane_addr + g * 128;
        const uint32_t o_addr = tmem_base + lane_addr + 256 + g * 128;
        const float c2 = args.scale_log2;
        // keys [0, see) of this part are visible to this row; see_w to the warp's first row, the fewest
        const int off = sp.nk - sp.nq;
        const int see = (args.causal ? min(sp.nk, qi + off + 1) : sp.nk) - kb;
        const int see_w = (args.causal ? min(sp.nk, w0 + off + 1) : sp.nk) - kb;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < ng && ok; ++j) {
            if (!wait_all(&s_full[g], j & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            uint32_t r[4][32];  // the score row, 128 columns; then P packed in r[0], r[1]
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, r[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) reg_fence32(r[c]);
            const bool edge = see_w < (j + 1) * AV_TILE;  // some column of the tile is hidden from some row
            const int lim = see - j * AV_TILE;
            auto sv = [&](int e) { return __uint_as_float(r[e >> 5][e & 31]); };
            float m4[4];
            auto row_max = [&](auto masked) {
                auto v = [&](int e) { return (!decltype(masked)::value || e < lim) ? sv(e) : -INFINITY; };
#pragma unroll
                for (int k = 0; k < 4; ++k) m4[k] = max3f(v(2 * k), v(2 * k + 1), -INFINITY);
#pragma unroll
                for (int e = 8; e < AV_TILE; e += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = max3f(m4[k], v(e + 2 * k), v(e + 2 * k + 1));
            };
            if (edge)
                row_max(std::true_type{});
            else
                row_max(std::false_type{});
            const float mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
            bool rescale = false;
            float alpha = 1.0f;
            if (j == 0) {
                m = mx;
            } else if ((mx - m) * c2 > AV_RESCALE_LOG2) {
                alpha = ex2_approx((m - mx) * c2);
                m = mx;
                l *= alpha;
                rescale = true;
            }
            // P = exp2(s c2 - m c2); column pair k packed as bf16x2 into word k (words <= 2k are read). A maximum of
            // -inf is no number to subtract: nothing was visible yet, or only scores of -inf (P = 0) and NaN (P, and
            // through it the sum, NaN: the maximum passes NaN over).
            const float2 c2v = make_float2(c2, c2);
            const float mb = m > -INFINITY ? -m * c2 : 0.0f;
            const float2 nmb = make_float2(mb, mb);
            float2 s4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) s4[k] = make_float2(0.0f, 0.0f);
            auto exp_pack = [&](auto masked) {
#pragma unroll
                for (int k = 0; k < AV_TILE / 2; ++k) {
                    const float2 x = fma2(make_float2(sv(2 * k), sv(2 * k + 1)), c2v, nmb);
                    float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    if (decltype(masked)::value) {
                        p.x = 2 * k < lim ? p.x : 0.0f;
                        p.y = 2 * k + 1 < lim ? p.y : 0.0f;
                    }
                    s4[k & 3] = add2(s4[k & 3], p);
                    r[k >> 5][k & 31] = pack_bf16x2(p.x, p.y);
                }
            };
            if (edge)
                exp_pack(std::true_type{});
            else
                exp_pack(std::false_type{});
            const float2 s2 = add2(add2(s4[0], s4[1]), add2(s4[2], s4[3]));
            l += s2.x + s2.y;
            tmem_st32(s_addr, r[0]);
            tmem_st32(s_addr + 32, r[1]);
            // Rows whose maximum rose: O_g *= alpha in TMEM before the next product adds to it.
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                for (int c = 0; c < NB; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_addr + c * 32, o);
                    tmem_wait_ld();
                    reg_fence32(o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                    tmem_st32(o_addr + c * 32, o);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[g]);
        }
        if (!JOIN && ok && rows_ok > 0) {
            const int row = sp.q0 + w0;
            if (lane < rows_ok)
                LSE[static_cast<long long>(head) * args.Tq + row + lane] =
                    l == 0.0f ? -INFINITY : fmaf(m, args.scale, logf(l));
            if (ng == 0) {
                av_store_zero_rows(0, NB, head * D, row, O, ldo, rows_ok, lane);
            } else if (wait_all(&o_full[g], 0)) {
                tc_fence_after();
                av_store_rows(o_addr, l == 0.0f ? 0.0f : 1.0f / l, 0, NB, sQ + g * T::BYTES + q * (NB * 2048), &tmO,
                              head * D, row, O, ldo, rows_ok, lane);
            }
        }
        if constexpr (JOIN) {
            if (ok && ng > 0) {
                ok = wait_all(&o_full[g], 0);
                tc_fence_after();
            }
            // Every row's maximum and sum go to all ranks. Chunk c (32 columns) of O_g is finished by rank
            // (g NB + c) % cluster; the others send it their rows, eight pieces of 16 bytes a row, into the rings:
            // [source rank][chunk of the owner][piece][128 rows].
            constexpr int CHUNK = 8 * AV_TILE;
            const int owned = (2 * NB + cluster - 1) / cluster;
            const int tile_row = q * 32 + lane;
            float2* stat = reinterpret_cast<float2*>(sQ) + g * AV_TILE + tile_row;  // [source rank][2][128]
            float4* recv = reinterpret_cast<float4*>(sK);
            __syncwarp();
            cluster_sync_all();  // every CTA of the cluster has used its tiles
            if (ok) {
                for (int s = 0; s < cluster; ++s)
                    st_cluster_v2(mapa_shared(smem_u32(stat + rank * 2 * AV_TILE), s), m, l);
                for (int c = 0; c < NB && ng > 0; ++c) {
                    const int id = g * NB + c, owner = id % cluster;
                    if (owner == rank) continue;
                    uint32_t o[32];
                    tmem_ld32(o_addr + c * 32, o);
                    tmem_ld_wait(o);
                    const uint32_t to =
                        mapa_shared(smem_u32(recv + (rank * owned + id / cluster) * CHUNK + tile_row), owner);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_cluster_v4(to + k * (AV_TILE * 16), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
            }
            __syncwarp();
            cluster_sync_all();
            if (ok && *abort_flag == 0u && rows_ok > 0) {
                float top = -INFINITY, sum = 0.0f;
                for (int s = 0; s < cluster; ++s) top = fmaxf(top, stat[s * 2 * AV_TILE].x);
                // a part's factor: its sum, NaN or 0, where that is NaN or the row saw none of its keys (whose O_g may
                // not have been computed)
                auto factor = [&](int s) {
                    const float2 part = stat[s * 2 * AV_TILE];
                    return part.x > -INFINITY && part.y == part.y ? ex2_approx((part.x - top) * c2) : part.y;
                };
                for (int s = 0; s < cluster; ++s) {
                    const float f = factor(s);
                    if (f != 0.0f) sum = fmaf(stat[s * 2 * AV_TILE].y, f, sum);
                }
                const int row = sp.q0 + w0 + lane;
                if (rank == 0 && lane < rows_ok)
                    LSE[static_cast<long long>(head) * args.Tq + row] =
                        sum == 0.0f ? -INFINITY : fmaf(top, args.scale, logf(sum));
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                for (int c = 0; c < NB; ++c) {
                    const int id = g * NB + c;
                    if (id % cluster != rank) continue;
                    uint32_t mine[32];
                    if (ng > 0) {
                        tmem_ld32(o_addr + c * 32, mine);
                        tmem_ld_wait(mine);
                    }
                    float o[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0.0f;
                    for (int s = 0; s < cluster; ++s) {
                        const float f = factor(s);
                        if (f == 0.0f) continue;
                        const float4* from = recv + (s * owned + id / cluster) * CHUNK + tile_row;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 v = s == rank ? make_float4(__uint_as_float(mine[4 * k]), __uint_as_float(mine[4 * k + 1]),
                                                                     __uint_as_float(mine[4 * k + 2]),
                                                                     __uint_as_float(mine[4 * k + 3]))
                                                       : from[k * AV_TILE];
                            o[4 * k] = fmaf(v.x, f, o[4 * k]);
                            o[4 * k + 1] = fmaf(v.y, f, o[4 * k + 1]);
                            o[4 * k + 2] = fmaf(v.z, f, o[4 * k + 2]);
                            o[4 * k + 3] = fmaf(v.w, f, o[4 * k + 3]);
                        }
                    }
                    if (lane < rows_ok) {
                        uint4* dst = reinterpret_cast<uint4*>(O + static_cast<long long>(row) * ldo + head * D + c * 32);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dst[k] = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                                pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                                pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                                pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                    }
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

// CTAs that share a pair of query tiles. The estimate, in iterations (a key tile each): a CTA costs 2.7 more than its
// own (its set-up, first loads and store), one of a cluster 5.4, 6.4 or 10 (the join too). Measured with 1, 2, 4, 8: one
// query on 16,384 keys, eight heads, d = 128, 175, 92, 50, 33 us; 4096 causal queries, d = 64, one head 45, 28, 19, 18,
// eight heads 46, 36, 58, 112; four prompts of 33 to 1025 queries, 20 heads, d = 96, 29, 43, 80, 179.
static int fwd_cluster(const AvArgs& a, int sms) {
    const double items = double(av_max_tiles(a.nseq, a.Tq, a.max_q, 2 * AV_TILE)) * a.heads;
    const double extra[4] = {2.7, 5.4, 6.4, 10.0};
    return av_cluster(items, ceil_div(a.max_k, AV_TILE), items * av_mean_keys(a), extra, 2, sms);
}

}  // namespace mptp

using namespace mptp;

extern "C" mp_status mp_attn_varlen_fwd(const mp_bf16* Q, const mp_bf16* K, const mp_bf16* V, mp_bf16* O, float* LSE,
                                        const int32_t* cu_q, const int32_t* cu_k, int nseq, int Tq, int Tk, int max_q,
                                        int max_k, int heads, int kv_heads, int d, long long ldq, long long ldk,
                                        long long ldv, long long ldo, int causal, float scale, uint32_t* d_status,
                                        void* stream) {
    mp_status st = av_check(nseq, Tq, Tk, max_q, max_k, heads, kv_heads, d, scale);
    if (st != MP_OK) return st;
    const long long qw = static_cast<long long>(heads) * d, kw = static_cast<long long>(kv_heads) * d;
    if (av_bad_pitch(ldq, qw) || av_bad_pitch(ldo, qw) || av_bad_pitch(ldk, kw) || av_bad_pitch(ldv, kw))
        return MP_ERR_UNSUPPORTED_SHAPE;
    if (nseq == 0 || max_q == 0) return MP_OK;
    if (!Q || !O || !LSE || !cu_q || !cu_k || (Tk > 0 && (!K || !V))) return MP_ERR_INVALID_ARG;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return MP_ERR_MISALIGNED;
    const void* words[] = {LSE, cu_q, cu_k, d_status};
    for (const void* p : words)
        if (reinterpret_cast<uintptr_t>(p) & 3u) return MP_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_device(&sms)) != MP_OK) return st;

    CUtensorMap tq, tk, tv, to;
    // Without keys the maps of K and V are never used: they take Q's.
    if (!av_tmap(&tq, Q, static_cast<int>(qw), Tq, ldq, d) || !make_tmap_bf16_out(&to, O, qw, Tq, ldo) ||
        !(Tk > 0 ? av_tmap(&tk, K, static_cast<int>(kw), Tk, ldk, d) && av_tmap(&tv, V, static_cast<int>(kw), Tk, ldv, d)
                 : av_tmap(&tk, Q, static_cast<int>(qw), Tq, ldq, d) && av_tmap(&tv, Q, static_cast<int>(qw), Tq, ldq, d)))
        return MP_ERR_CUDA;
    const AvArgs a = av_args(cu_q, cu_k, nseq, Tq, Tk, max_q, max_k, heads, kv_heads, causal ? 1 : 0, scale, d_status);
    const long long blocks = av_max_tiles(nseq, Tq, max_q, 2 * AV_TILE) * heads;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(O);
    const int cluster = fwd_cluster(a, sms);
    auto launch = [&](auto alone, auto joined, size_t smem) {
        return av_launch(cluster > 1 ? joined : alone, blocks * cluster, cluster, smem, s, tq, tk, tv, to, o, ldo, LSE, cluster, a);
    };
    const cudaError_t e =
        d == 64   ? launch(attn_varlen_fwd_kernel<64, false>, attn_varlen_fwd_kernel<64, true>, AvFwdCfg<64>::SMEM)
        : d == 96 ? launch(attn_varlen_fwd_kernel<96, false>, attn_varlen_fwd_kernel<96, true>, AvFwdCfg<96>::SMEM)
                  : launch(attn_varlen_fwd_kernel<128, false>, attn_varlen_fwd_kernel<128, true>, AvFwdCfg<128>::SMEM);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
