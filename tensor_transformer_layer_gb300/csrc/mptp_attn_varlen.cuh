// What the kernels of the packed attention (forward, query gradient, key and value gradients) share:
// the sequences' spans, tile sizes, tile loads, the clearing of rows behind a sequence's end, and the
// store of a warp's 32 rows.
//
// Tiles are 128 rows of D columns, loaded as D/32 boxes of 32 columns with the 64-byte swizzle. The
// same tile serves as a K-major operand (D is the summed dimension) and as an MN-major one (its rows
// are summed), so nothing is transposed.
#pragma once

#include "mptp_gemm.cuh"
#include "mptp_internal.h"

namespace mptp {

constexpr uint32_t DEV_SEQ_RANGE = 0x4u;
constexpr int AV_TILE = 128;     // rows per tile
constexpr int AV_MAX_CLUSTER = 8;
constexpr int AV_THREADS = 384;  // warpgroup 0: loads, MMA, helpers; 1 and 2: softmax

template <int D>
struct AvTile {
    static_assert(D == 64 || D == 96 || D == 128, "head width");
    static constexpr int NB = D / 32;              // 32-column boxes
    static constexpr int BOX = AV_TILE * 64;       // bytes of one box
    static constexpr int BYTES = NB * BOX;         // bytes of one tile
    // Registers a thread in warpgroup 0 and in the softmax warpgroups (setmaxnreg); the launch gives
    // 384 x 168.
    static constexpr int REGS_CTRL = 88;
    static constexpr int REGS_SOFTMAX = 208;
    static_assert(128 * REGS_CTRL + 256 * REGS_SOFTMAX <= AV_THREADS * 168, "register split");
};

struct AvArgs {
    const int32_t* cu_q;
    const int32_t* cu_k;
    int nseq, Tq, Tk, max_q, max_k;
    int heads, kv_heads, group;  // group = heads / kv_heads
    int causal;
    float scale, scale_log2;     // scale_log2 = scale * log2(e)
    uint32_t* status;
    unsigned long long budget_ns;
};

// Rows of one sequence. A span that is not inside the tensors or longer than the caller's maximum is
// reported and left out (nothing of it is read or written).
struct AvSpan {
    int q0, nq, k0, nk;
};
__device__ __forceinline__ AvSpan av_span(const AvArgs& a, int seq) {
    const int q0 = a.cu_q[seq], q1 = a.cu_q[seq + 1], k0 = a.cu_k[seq], k1 = a.cu_k[seq + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk || q1 - q0 > a.max_q || k1 - k0 > a.max_k) {
        if (threadIdx.x < 32 && a.status) atomicOr(a.status, DEV_SEQ_RANGE);
        return {0, 0, 0, 0};
    }
    return {q0, q1 - q0, k0, k1 - k0};
}

// The sequence and tile at place `item` of the order in which CTAs take them; false where there are no so many. A
// tile has ROWS rows, queries (OF_QUERIES) or keys. The sequences with the longest other side come first, of each the
// tiles that meet most of it first, so that a launch ends with small work; sequences beyond 32 follow by 32. Each
// warp finds the place by itself, a lane a sequence. (A grid of every sequence by the longest one's tiles needs no
// search, but a CTA that finds no tile costs 0.6 to 1.1 us with its launch and shared memory: 64 sequences of 128
// tokens with a maximum of 2432 took 101, 160 and 54 us in the three kernels, and take 49, 53 and 24. The order by
// work exactly, a search over all sequences' tiles, lost 1 to 2 us a CTA to the search.) The walk over the offsets is a step
// for every 32 sequences before the tile's: 512, 1024 and 4096 sequences of 8 tokens, eight heads on two, d = 64, take the
// forward 170, 405 and 3180 us, where the CTAs alone would grow from 170 to 1360.
template <int ROWS, bool OF_QUERIES>
__device__ __forceinline__ bool av_pick(const AvArgs& a, int item, AvSpan& sp, int& tile) {
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < a.nseq; base += 32) {
        const int m = min(32, a.nseq - base);
        const AvSpan s = lane < m ? av_span(a, base + lane) : AvSpan{0, 0, 0, 0};
        const int tiles = ((OF_QUERIES ? s.nq : s.nk) + ROWS - 1) / ROWS;
        const int other = OF_QUERIES ? s.nk : s.nq;
        const int all = __reduce_add_sync(0xffffffffu, tiles);
        if (item >= all) {
            item -= all;
            continue;
        }
        int first = 0;  // tiles of the sequences before the lane's
        for (int j = 0; j < m; ++j) {
            const int v = __shfl_sync(0xffffffffu, tiles, j), w = __shfl_sync(0xffffffffu, other, j);
            if (w > other || (w == other && j < lane)) first += v;
        }
        const int at = item - first;
        const bool here = at >= 0 && at < tiles;
        // Sums of one lane's value leave it in a uniform register, as the loops over tiles want it: with shuffles in
        // their place the key gradients of 4096 tokens and 19 heads took 220 us at D = 128, with them 213 at the time.
        auto value = [&](int v) { return __reduce_add_sync(0xffffffffu, here ? v : 0); };
        sp = {value(s.q0), value(s.nq), value(s.k0), value(s.nk)};
        tile = value(OF_QUERIES ? tiles - 1 - at : at);
        return true;
    }
    return false;
}

// A place in a ring of N tiles, counted along by the warp that issues the products.
template <int N>
struct AvRing {
    int st = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) {
            st = 0;
            ph ^= 1u;
        }
    }
};

// One tile (rows from `row`, head `head` of the matrix) into shared memory, counted on `bar`: D/32 boxes by one
// load.
template <int D>
__device__ __forceinline__ void av_load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head, int row) {
    using C = AvTile<D>;
    mbar_arrive_expect_tx(bar, C::BYTES);
    tma_load_3d(dst, map, bar, 0, row, head * C::NB);
}

// A wait budget of zero stands for loads that never arrive, in every CTA or, of a cluster, in its last one: its first
// tiles are not asked for, so that its waits do run out.
__device__ __forceinline__ bool av_starved(const AvArgs& a, int rank, int cluster) {
    return a.budget_ns == 0 && rank == cluster - 1;
}

// The part that the loading and issuing warps take in a cluster's join: its two barriers. Between them a CTA that gave up
// makes the others of its cluster give up too: it sends them nothing, and what they would add in its place is old tiles.
__device__ __forceinline__ void av_join_barriers(volatile uint32_t* abort_flag, int cluster, int warp, int lane) {
    __syncwarp();
    cluster_sync_all();
    if (warp == 0 && lane < cluster && *abort_flag != 0u)
        st_cluster_b32(mapa_shared(smem_u32(const_cast<uint32_t*>(abort_flag)), lane), 1u);
    __syncwarp();
    cluster_sync_all();
}

// One warp clears rows [from, 128) of a tile in shared memory. A tile that reaches past its sequence
// holds the next one's rows: their products with zero weights would still carry infinities and NaN.
template <int D>
__device__ __forceinline__ void av_clear_rows(uint8_t* tile, int from, int lane) {
    using C = AvTile<D>;
    for (int i = from * 4 + lane; i < AV_TILE * 4; i += 32)
#pragma unroll
        for (int c = 0; c < C::NB; ++c)
            *reinterpret_cast<uint4*>(tile + c * C::BOX + i * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();  // the tensor core reads them through the async proxy
    __syncwarp();
}

// Chunks [c0, c1) (32 columns each) of a warp's 32 accumulator rows, times f, as bf16: through shared
// memory and TMA where all 32 rows belong to the sequence (rows_ok = 32), else row by row. `acc` is the
// warp's TMEM address, `stg` its 2 KB boxes, one per chunk of the tile. A row whose f is 0 saw no key and is
// zero: its accumulators may hold NaN, zero weights times infinities among the keys of its tile.
__device__ __forceinline__ void av_store_rows(uint32_t acc, float f, int c0, int c1, uint8_t* stg,
                                              const CUtensorMap* map, int col, int row, __nv_bfloat16* out,
                                              long long ld, int rows_ok, int lane) {
    const int sw = (lane >> 1) & 3;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
        uint32_t o[32];
        tmem_ld32(acc + c * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
        uint4 w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v)
            w[v] = make_uint4(pack_bf16x2(__uint_as_float(o[8 * v]) * f, __uint_as_float(o[8 * v + 1]) * f),
                              pack_bf16x2(__uint_as_float(o[8 * v + 2]) * f, __uint_as_float(o[8 * v + 3]) * f),
                              pack_bf16x2(__uint_as_float(o[8 * v + 4]) * f, __uint_as_float(o[8 * v + 5]) * f),
                              pack_bf16x2(__uint_as_float(o[8 * v + 6]) * f, __uint_as_float(o[8 * v + 7]) * f));
        if (f == 0.0f) {
#pragma unroll
            for (int v = 0; v < 4; ++v) w[v] = make_uint4(0u, 0u, 0u, 0u);
        }
        if (rows_ok >= 32) {
            uint8_t* r = stg + c * 2048 + lane * 64;
#pragma unroll
            for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(r + ((v ^ sw) << 4)) = w[v];
        } else if (lane < rows_ok) {
            uint4* r = reinterpret_cast<uint4*>(out + static_cast<long long>(row + lane) * ld + col + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) r[v] = w[v];
        }
    }
    if (rows_ok >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) tma_store_2d(map, stg + c * 2048, col + c * 32, row);
            bulk_commit_group();
            bulk_wait_group_read<0>();  // the staging is read before the CTA exits; the grid's end has it written
        }
        __syncwarp();
    }
}

// The same rows as zeros.
__device__ __forceinline__ void av_store_zero_rows(int c0, int c1, int col, int row, __nv_bfloat16* out, long long ld,
                                                   int rows_ok, int lane) {
    if (lane >= rows_ok) return;
    uint4* r = reinterpret_cast<uint4*>(out + static_cast<long long>(row + lane) * ld + col);
    for (int i = c0 * 4; i < c1 * 4; ++i) r[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Key tiles that a tile of queries [i0, i0 + 128) of a sequence sees (causal: the last query sees the
// last key).
__device__ __forceinline__ int av_key_tiles(const AvSpan& s, int i0, int causal) {
    if (i0 >= s.nq) return 0;
    int keys = s.nk;
    if (causal) {
        const int last = min(i0 + AV_TILE, s.nq) + (s.nk - s.nq);
        keys = min(keys, last);
    }
    return keys > 0 ? (keys + AV_TILE - 1) / AV_TILE : 0;
}

// 16-bit A operand of a TMEM product: 16 rows' worth (8 columns) of step k. Each softmax warpgroup
// writes its 64 columns' values, packed, over the first half of its own 64 fp32 columns.
__device__ __forceinline__ uint32_t av_a_step(uint32_t base, int k) { return base + (k >> 2) * 64 + (k & 3) * 8; }

inline bool av_tmap(CUtensorMap* m, const void* base, int cols, int rows, long long ld, int d) {
    return make_tmap_bf16_sw64_3d(m, base, cols, rows, ld, AV_TILE, d / 32);
}

// Tiles of `rows` rows that sequences of no more than T rows together, `longest` each, can have.
inline long long av_max_tiles(int nseq, int T, int longest, int rows) {
    const long long each = static_cast<long long>(nseq) * ceil_div(longest, rows), all = T / rows + static_cast<long long>(nseq);
    return each < all ? each : all;
}

// Sizes, pitches and pointers that the forward and the backward refuse alike.
inline mp_status av_check(int nseq, int Tq, int Tk, int max_q, int max_k, int heads, int kv_heads, int d, float scale) {
    if (nseq < 0 || Tq < 0 || Tk < 0 || max_q < 0 || max_k < 0 || heads <= 0 || kv_heads <= 0 || d <= 0 ||
        !(scale > 0.0f) || !(scale <= 3.0e38f))
        return MP_ERR_INVALID_ARG;
    if (heads % kv_heads != 0 || (d != 64 && d != 96 && d != 128) || max_q > Tq || max_k > Tk ||
        static_cast<long long>(heads) * d > 0x3fffffff)
        return MP_ERR_UNSUPPORTED_SHAPE;
    // CTAs of the largest launches: the tiles that can exist, of every head, in the largest clusters
    const long long most = 0x7fffffffLL / AV_MAX_CLUSTER;
    if (av_max_tiles(nseq, Tq, max_q, AV_TILE) > most / heads || av_max_tiles(nseq, Tk, max_k, AV_TILE) > most / kv_heads)
        return MP_ERR_UNSUPPORTED_SHAPE;
    return MP_OK;
}
inline bool av_bad_pitch(long long ld, long long row) { return ld < row || ld % 8 != 0 || ld > (1LL << 36); }

inline AvArgs av_args(const int32_t* cu_q, const int32_t* cu_k, int nseq, int Tq, int Tk, int max_q, int max_k,
                      int heads, int kv_heads, int causal, float scale, uint32_t* status) {
    AvArgs a{};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.nseq = nseq;
    a.Tq = Tq;
    a.Tk = Tk;
    a.max_q = max_q;
    a.max_k = max_k;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.group = heads / kv_heads;
    a.causal = causal;
    a.scale = scale;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.status = status;
    a.budget_ns = wait_budget_ns();
    return a;
}

// Key tiles that a query tile sees on average, estimated: the lengths are on the device, so the sum over the sequences is
// taken between that of equal ones and that of the longest.
inline double av_mean_keys(const AvArgs& a) {
    const double keys = 0.5 * (a.max_k + double(a.Tk) / a.nseq);
    const double hidden = a.causal ? 0.25 * (a.max_q + double(a.Tq) / a.nseq) : 0.0;
    return (keys > hidden ? keys - hidden : 0.0) / AV_TILE + 0.5;
}

// CTAs that share an item: 1, 2, 4 or 8, by the larger of the longest CTA and of all the work over the SMs that clusters of
// the size can use. `items` CTAs without sharing, the longest of `longest` iterations, all of `total`; extra[i]: what a
// CTA costs beside its iterations in clusters of 2^i; part_least: iterations that the longest keeps at least.
inline int av_cluster(double items, double longest, double total, const double (&extra)[4], int part_least, int sms) {
    const double usable[4] = {1.0, 1.0, 0.95, 0.79};  // of the SMs: 152, 152, 144, 120
    int best = 1;
    double least = 0.0;
    for (int i = 0; i < 4; ++i) {
        const int c = 1 << i;
        if (c > 1 && longest < part_least * c) break;
        const double even = (total + items * c * extra[i]) / (sms * usable[i]);
        const double part = longest / c + extra[i];
        const double est = even > part ? even : part;
        if (i == 0 || est < 0.9 * least) {
            best = c;
            least = est;
        }
    }
    return best;
}

// `blocks` CTAs in clusters of `cluster`.
template <typename Kern, typename... Args>
inline cudaError_t av_launch(Kern kern, long long blocks, int cluster, size_t smem, cudaStream_t s, Args... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(AV_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mptp
