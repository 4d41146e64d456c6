// Host helpers of the feed-forward blocks (GeLU and gated): GEMM problems, tile and schedule
// choices, and the launches that both blocks' backward passes share.
#pragma once

#include <cstdlib>
#include <cstring>

#include "mptp_gemm.cuh"
#include "mptp_gemm_split.cuh"
#include "mptp_internal.h"

namespace mptp {

inline mp_status check_mlp_shape(int T, int h, int f, int t) {
    if (T < 0 || h <= 0 || f <= 0 || t < 1) return MP_ERR_INVALID_ARG;
    if (h % 64 != 0 || f % t != 0 || (f / t) % 64 != 0) return MP_ERR_UNSUPPORTED_SHAPE;
    return MP_OK;
}

inline mp_status check_shard_range(int t, int s0, int n) {
    if (s0 < 0 || n < 1 || s0 > t - n) return MP_ERR_INVALID_ARG;
    return MP_OK;
}

// One GEMM of a launch: C[M, N] over K blocks [kb_begin, kb_end). a_bytes / b_bytes
// are the sizes of the A (M side) and B (N side) operands, for the unit order.
inline ProbInfo problem(int M, int N, int bn, int kb_begin, int kb_end, bool a_mn, bool b_mn, double a_bytes,
                        double b_bytes) {
    ProbInfo p{};
    p.M = M;
    p.N = N;
    p.num_m_blocks = ceil_div(M, 2 * BM);  // 256-row blocks: one per CTA-pair tile
    p.num_units = p.num_m_blocks * ceil_div(N, bn);
    p.n_fastest = n_fastest_order(a_bytes, b_bytes);
    p.kb_begin = kb_begin;
    p.kb_end = kb_end;
    p.a_mn = a_mn ? 1 : 0;
    p.b_mn = b_mn ? 1 : 0;
    return p;
}

// Backward schedule of K4, K5a, K5b: MPTP_BWD_SCHEDULE = "serial" | "overlap"; unset or
// anything else picks the side-by-side schedule when its estimated makespan is at least
// 6 % below the serial one. Measured on GB300 over h in {768..3072}, T in {512..8192}:
// it wins 1-50 % where the estimate says >= 7 %, and loses up to 5 % at h = 3072 with
// T >= 4096 (estimate <= 5.5 %), where three GEMMs' operand panels crowd L2.
enum class BwdSchedule { Auto, Serial, Overlap };
inline BwdSchedule bwd_schedule() {
    const char* v = std::getenv("MPTP_BWD_SCHEDULE");
    if (v != nullptr && std::strcmp(v, "serial") == 0) return BwdSchedule::Serial;
    if (v != nullptr && std::strcmp(v, "overlap") == 0) return BwdSchedule::Overlap;
    return BwdSchedule::Auto;
}

// Cost of one output tile in K-block times: its K blocks plus about two for the epilogue.
constexpr int EPI_KB = 2;
// What a tile costs at least, its epilogue's time (2.3 us of stores): with one K block, products of 64 tokens, a plan by
// K blocks left 432 tiles to seven pairs beside a long product, 144 us.
constexpr int TILE_MIN_KB = 9;
inline int tile_cost(const GemmArgs& a) {
    const int cost = a.pr.kb_end - a.pr.kb_begin + EPI_KB;
    return cost > TILE_MIN_KB ? cost : TILE_MIN_KB;
}

// Epilogue warps of K1 and K3 (GeLU, GeLU'). A launch's last tile is epilogued after its last
// MMA with nothing to hide behind: with few K blocks per CTA pair (the layer at T = 2048,
// h = 1536: 72 a pair) eight warps halve that tail (K3's 10.6 -> 6.3 us, K1's 5.4 -> 4.0 us;
// the step -1 %), while on long launches four measured 0.2-0.8 % faster (fewer warps beside the
// MMA issuer). The store-only GEMMs keep four: eight were 1 % slower there.
constexpr int SHORT_LAUNCH_KB = 256;  // K blocks a pair runs, at most, for eight epilogue warps

template <int EPI>
inline cudaError_t launch_gelu_epi(const TmapSet& m, const GemmArgs& a, int sms, cudaStream_t s) {
    const int pairs = resident_pairs<256, EPI, 4>(sms);
    const bool short_launch = ceil_div(a.pr.num_units, pairs) * (a.pr.kb_end - a.pr.kb_begin) <= SHORT_LAUNCH_KB;
    return short_launch ? launch_gemm_tc<256, EPI, 8>(m, a, sms, s) : launch_gemm_tc<256, EPI, 4>(m, a, sms, s);
}

// Tile width of K4 (dX = dU A^T, N = h, B operand K-major). 224-wide tiles cut h = 3072
// into 14 column units instead of 12, so T = 4096 gives 224 units: 2.95 rounds of 76 CTA
// pairs, against 2.53 rounds of 256-wide tiles whose last round leaves half the pairs idle.
constexpr int K4_BN = 224;

// Split-K for the row-parallel GEMMs (K2, K4) when their output tiles do not fill the chip:
// the two CTA pairs of a cluster share a 256-wide tile, each over half of the shard-ordered K
// range, and the partials are summed on chip (mptp_gemm_split.cuh). Costs in K-block times:
// one pair per tile, `bn` wide, takes rounds x L x bn / 256; two pairs take
// rounds x ceil(L / 2) plus about SPLIT_HOP_KB for the on-chip sum. The split is taken when it
// is at least 10 % cheaper and each pair keeps at least 16 K blocks (T = 2048, h = 3072: 96
// tiles on 36 clusters, 292 against 384; the forward 5.6 % faster). Measured and not kept:
// 128-wide split tiles (at T = 2048, h = 1536 the forward took 81 us against 68 us unsplit), and
// clusters of three or four pairs, which fit only 23 or 15 at a time on the 152-SM GB300 and beat
// two pairs at no layer shape of the Megatron-LM sweep.
constexpr int SPLIT_PAIRS = 2;
constexpr int SPLIT_HOP_KB = 4;
constexpr int SPLIT_MIN_KB = 16;

inline long long tiles_of(int M, int N, int bn) { return static_cast<long long>(ceil_div(M, 2 * BM)) * ceil_div(N, bn); }

// True when the split kernel should run this GEMM (M x N, L K blocks) instead of the
// single-pair kernel with BN1-wide tiles.
template <int BN1>
inline bool use_split(int M, int N, int L, int sms) {
    const int pairs = resident_pairs<BN1, EPI_STORE, 4>(sms);
    const int clusters = resident_split_clusters<256, SPLIT_PAIRS>(sms);
    if (clusters <= 0 || L < SPLIT_MIN_KB * SPLIT_PAIRS) return false;
    const long long one = (tiles_of(M, N, BN1) + pairs - 1) / pairs * L * BN1;  // x 1/256 K-block times
    const long long two =
        ((tiles_of(M, N, 256) + clusters - 1) / clusters * ceil_div(L, SPLIT_PAIRS) + SPLIT_HOP_KB) * 256;
    return two * 10 <= one * 9;
}

inline GemmArgs launch_args(uint32_t* status) {
    GemmArgs a{};
    a.tiles_per_unit = 1;
    a.status = status;
    a.budget_ns = wait_budget_ns();
    return a;
}

// K4 with tiles of `bn` columns (224 or 256; outputs do not depend on it).
inline cudaError_t launch_k4(int bn, const TmapSet& m, const GemmArgs& a, int sms, cudaStream_t s, int max_pairs = 0) {
    return bn == K4_BN ? launch_gemm_tc<K4_BN, EPI_STORE, 4>(m, a, sms, s, max_pairs)
                       : launch_gemm_tc<256, EPI_STORE, 4>(m, a, sms, s, max_pairs);
}

// dX, dA and dB of a block's backward (K4, K5a, K5b): one after another, or side by side on
// disjoint CTA pairs. m4 / a4 hold K4 with bn4-wide tiles (K4_BN or 256) over the K-major weight
// W [h, ldw], whose operand map is rebuilt for 256-wide tiles where K4 runs split.
inline mp_status launch_grad_gemms(TmapSet& m4, GemmArgs& a4, int bn4, const mp_bf16* W, int ldw, const TmapSet& m5,
                                   const GemmArgs& a5, const TmapSet& m6, const GemmArgs& a6, int sms,
                                   cudaStream_t s) {
    const int h = a4.pr.N;
    // Every output tile is computed by the same K-loop whichever pairs run it, so both
    // schedules give bitwise identical results.
    const int pairs = resident_pairs<256, EPI_STORE, 4>(sms);
    const int units[3] = {a4.pr.num_units, a5.pr.num_units, a6.pr.num_units};
    const int cost[3] = {tile_cost(a4), tile_cost(a5), tile_cost(a6)};
    int split[3] = {pairs, pairs, pairs};
    const BwdSchedule mode = bwd_schedule();
    bool overlap = false;
    if (mode != BwdSchedule::Serial && pairs >= 3) {
        const long long side = split_pairs(pairs, 3, units, cost, split);
        overlap = mode == BwdSchedule::Overlap || side * 100 <= serial_makespan(pairs, 3, units, cost) * 94;
    }
    if (overlap) {
        std::lock_guard<std::mutex> lock(side_stream_mutex());
        SideStreams* ss = side_streams(s);
        if (ss != nullptr) {
            bool ok = cudaEventRecord(ss->fork, s) == cudaSuccess &&
                      cudaStreamWaitEvent(ss->s[0], ss->fork, 0) == cudaSuccess &&
                      cudaStreamWaitEvent(ss->s[1], ss->fork, 0) == cudaSuccess;
            if (!ok) return MP_ERR_CUDA;
            ok = launch_k4(bn4, m4, a4, sms, s, split[0]) == cudaSuccess;
            ok = launch_gemm_tc<256, EPI_STORE, 4>(m5, a5, sms, ss->s[0], split[1]) == cudaSuccess && ok;
            ok = launch_gemm_tc<256, EPI_STORE, 4>(m6, a6, sms, ss->s[1], split[2]) == cudaSuccess && ok;
            // Join even after a failed launch, so the caller's stream never runs ahead of the side streams.
            for (int i = 0; i < 2; ++i)
                ok = cudaEventRecord(ss->join[i], ss->s[i]) == cudaSuccess &&
                     cudaStreamWaitEvent(s, ss->join[i], 0) == cudaSuccess && ok;
            return ok ? MP_OK : MP_ERR_CUDA;
        }
    }
    const int L4 = a4.pr.kb_end - a4.pr.kb_begin;
    const bool split4 = bn4 == K4_BN ? use_split<K4_BN>(a4.pr.M, h, L4, sms) : use_split<256>(a4.pr.M, h, L4, sms);
    if (split4) {
        // The split kernel's 256-wide tiles: B boxes of 128 rows per CTA.
        if (!make_tmap_bf16(&m4.b, W, ldw, h, ldw, 64, 128)) return MP_ERR_CUDA;
        a4.pr.num_units = a4.pr.num_m_blocks * ceil_div(h, 256);
    }
    if ((split4 ? launch_gemm_split<256, SPLIT_PAIRS>(m4, a4, sms, s) : launch_k4(bn4, m4, a4, sms, s)) != cudaSuccess ||
        launch_gemm_tc<256, EPI_STORE, 4>(m5, a5, sms, s) != cudaSuccess ||
        launch_gemm_tc<256, EPI_STORE, 4>(m6, a6, sms, s) != cudaSuccess)
        return MP_ERR_CUDA;
    return MP_OK;
}

}  // namespace mptp
