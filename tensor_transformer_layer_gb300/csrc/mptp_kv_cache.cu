// Entry points of the 8-bit cache of keys and values: mp_kv_cache_write, mp_kv_cache_read.
//
// Write. Of a page's new rows and a head: amax, then the scale s, the smallest power of two with amax <= 448 s (448
// is the largest e4m3 value; not below 2^-100), then codes rn(x / s). A power of two loses nothing: e4m3 is a floating
// type, so a scale within a factor of two changes no relative error but at the bottom of its range, x / s is exact, and
// a part-filled page whose new rows need a larger scale keeps its old codes exact too (they are shifted, and rounded
// again only where they become subnormal). The codes follow from the inputs bit for bit.
//
// Read. code * scale, rounded to bf16 (exact for scales that a write left, short of bf16's own subnormals).
//
// Both are bound by memory: 2 bytes in and 1 out for each element, or 1 in and 2 out. A group of threads takes a unit, the rows
// of one page, head and kind (keys or values), all of them in registers at once, so that the amax and the codes come from one
// read. A block finds its page once and walks a share of its units; a write's come through shared memory two units ahead,
// each thread's own places, at offsets that are the same in every unit (15.5 k tokens of 8 heads of 96 18.6 us, with the next unit in
// registers and its addresses anew 19.5; 156 k 122 and 139).
// Measured: a write of 156 k tokens 5.9 TB/s, of 15.5 k 3.8 (three reads in a row before the first code, then eight steps in blocks
// that are all there at once); a read of 102 k tokens of 8 heads of 128 97 us, 6.5 TB/s, 96 % of a copy's rate.
#include <type_traits>

#include "mptp_kv_cache.cuh"
#include "mptp_launch.cuh"

namespace mptp {

// Threads of a block, and blocks that a launch is split into where it has so many units.
constexpr int KV_WRITE_THREADS = 128;  // or twice as many, where a unit's vectors fill them
constexpr int KV_WRITE_BLOCKS = 152 * 3;
// A block's units in flight, and the one in hand (two: 18.4 and 121 us for the sizes above; 29 k tokens 32.4, three 30.2).
constexpr int KV_WRITE_STAGES = 3;
constexpr int KV_READ_THREADS = 256;
constexpr int KV_READ_BLOCKS = 152 * 24;

struct KvRows {
    const __nv_bfloat16* in[2];  // write: new keys and values
    __nv_bfloat16* out[2];       // read
    long long ld[2];
    uint32_t ld16[2];  // the same in 16-byte pieces
    const int32_t* cu;     // [nseq + 1]
    const int32_t* start;  // [nseq] or null: zeros
    int nseq, T, max_n;
    int per_seq;  // pages a sequence may touch: page `item` is that of sequence item / per_seq. 0: found by a search
    int group_shift;     // log2 of the threads of a unit: 32 to a block's
    int splits;          // blocks that share a page's units
    int held;            // write: vectors of a thread
    uint32_t per_row;    // ceil(2^32 / (d / 8)): v * per_row >> 32 is the row of vector v (exact for v < 2^16, d <= 256)
    uint32_t* status;
};

// The rows of one page that a call touches.
struct KvPage {
    int row;      // packed row of the first
    int id;       // page in the pool
    int a, b;     // slots [a, b)
};

// A sequence that breaks the rules is reported and left out.
__device__ __forceinline__ void kv_span(const KvRows& r, const KvPool& p, int seq, int& row0, int& first, int& n) {
    row0 = r.cu[seq];
    const int end = r.cu[seq + 1];
    first = r.start != nullptr ? r.start[seq] : 0;
    n = end - row0;
    if (row0 < 0 || end < row0 || end > r.T || n > r.max_n || first < 0 ||
        static_cast<long long>(first) + n > static_cast<long long>(p.max_pages) * p.page) {
        if (r.status != nullptr) atomicOr(r.status, KV_SEQ_RANGE);
        n = 0;
    }
}
__device__ __forceinline__ int kv_touched(const KvPool& p, int first, int n) {
    return n > 0 ? ((first + n - 1) >> p.page_shift) - (first >> p.page_shift) + 1 : 0;
}

// The `item`-th page that the call touches; false where there are no so many. With few pages a sequence (per_seq) the
// place follows from the number; else each warp searches, a lane a sequence.
__device__ __forceinline__ bool kv_pick(const KvRows& r, const KvPool& p, int item, KvPage& out) {
    int seq = -1, row0 = 0, first = 0, n = 0, at = 0;
    if (r.per_seq > 0) {
        seq = item / r.per_seq;
        at = item % r.per_seq;
        if (seq >= r.nseq) return false;
        kv_span(r, p, seq, row0, first, n);
        if (at >= kv_touched(p, first, n)) return false;
    } else {
        const int lane = threadIdx.x & 31;
        for (int base = 0; base < r.nseq; base += 32) {
            if (base + lane < r.nseq) kv_span(r, p, base + lane, row0, first, n);
            else n = 0;
            const int mine = kv_touched(p, first, n);
            int upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += v;
            }
            const int all = __shfl_sync(0xffffffffu, upto, 31);
            if (item >= all) {
                item -= all;
                continue;
            }
            const int who = __ffs(__ballot_sync(0xffffffffu, item < upto)) - 1;
            seq = base + who;
            at = item - __shfl_sync(0xffffffffu, upto - mine, who);
            row0 = __shfl_sync(0xffffffffu, row0, who);
            first = __shfl_sync(0xffffffffu, first, who);
            n = __shfl_sync(0xffffffffu, n, who);
            break;
        }
        if (seq < 0) return false;
    }
    const int logical = (first >> p.page_shift) + at;
    const int begin = logical << p.page_shift;
    out.a = max(first - begin, 0);
    out.b = min(first + n - begin, p.page);
    out.row = row0 + (begin + out.a - first);
    out.id = p.table[static_cast<long long>(seq) * p.max_pages + logical];
    if (out.id < 0 || out.id >= p.pages) {
        if (r.status != nullptr) atomicOr(r.status, KV_PAGE_RANGE);
        return false;
    }
    return true;
}

// The scale that an amax (a bf16 value, finite) needs, as its exponent: the smallest e with amax <= 448 * 2^e.
__device__ __forceinline__ int kv_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
    return max(e, -100);
}
__device__ __forceinline__ float kv_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ float kv_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float kv_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Largest finite magnitude of two bf16 values and `m`.
__device__ __forceinline__ float kv_amax_finite(uint32_t w, float m) {
    const float a = fabsf(kv_lo(w)), b = fabsf(kv_hi(w));
    m = a < __int_as_float(0x7f800000) ? fmaxf(m, a) : m;
    return b < __int_as_float(0x7f800000) ? fmaxf(m, b) : m;
}
// Largest magnitudes of pairs of bf16 values, infinities among them; NaN is passed over.
__device__ __forceinline__ __nv_bfloat162 kv_amax2(uint32_t w, __nv_bfloat162 m) {
    return __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
}

// Two values as codes; inv: the scale's inverse twice. Their product is exact in bf16 but for magnitudes below 2^-126, whose code
// is zero in any case. e4m3 has no infinity: one (INF: there are some) becomes NaN, so that whoever reads it sees it.
template <bool INF>
__device__ __forceinline__ uint32_t kv_quant2(uint32_t w, __nv_bfloat162 inv) {
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), inv);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&x);
    float a = kv_lo(u), b = kv_hi(u);
    if constexpr (INF) {
        if (isinf(a)) a = __int_as_float(0x7fffffff);
        if (isinf(b)) b = __int_as_float(0x7fffffff);
    }
    return float2_to_e4m3x2(a, b);
}
template <bool INF>
__device__ __forceinline__ uint2 kv_quant8(const uint4& x, __nv_bfloat162 inv) {
    return make_uint2(kv_quant2<INF>(x.x, inv) | kv_quant2<INF>(x.y, inv) << 16,
                      kv_quant2<INF>(x.z, inv) | kv_quant2<INF>(x.w, inv) << 16);
}

// Four codes times a ratio <= 1, rounded again.
__device__ __forceinline__ uint32_t kv_requant4(uint32_t c, float ratio) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(c)), b = f16x2_to_float2(e4m3x2_hi_to_f16x2(c));
    return float2_to_e4m3x2(a.x * ratio, a.y * ratio) | float2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
}

// 16 or 4 bytes of a thread into its own place in shared memory; zeros where they are not taken.
__device__ __forceinline__ void kv_copy16(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void kv_copy4(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}

// NV: vectors of eight elements that a thread holds at most.
template <int NV, int THREADS>
struct KvStage {
    static constexpr int VECTORS = NV * THREADS * 16;
    static constexpr int BYTES = VECTORS + THREADS * 4;  // then the page's scale so far
    static constexpr int SMEM = KV_WRITE_STAGES * BYTES;
};
template <int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const KvRows r, const KvPool p) {
    using S = KvStage<NV, THREADS>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red[THREADS / 32];
    const int group = 1 << r.group_shift, per_cta = THREADS >> r.group_shift;
    const int item = blockIdx.x / r.splits, split = blockIdx.x % r.splits;
    const int tid = threadIdx.x & (group - 1), wide = p.d >> 3;
    grid_dependency_wait();
    grid_launch_dependents();
    KvPage at;
    if (!kv_pick(r, p, item, at)) return;
    const int count = (at.b - at.a) * wide;
    // Over the threads of the unit, the same in all of them.
    auto largest = [&](float m) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (group > 32) {
            __syncthreads();
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
            __syncthreads();
            const int w0 = threadIdx.x >> r.group_shift << (r.group_shift - 5);
            for (int k = 0; k < group >> 5; ++k) m = fmaxf(m, red[w0 + k]);
        }
        return m;
    };
    const uint32_t ring = smem_u32(smem) + threadIdx.x * 16;
    // The thread's vectors within a unit, the same in every one.
    uint32_t rows[NV], cols[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int v = tid + (k << r.group_shift);
        rows[k] = __umulhi(v, r.per_row);
        cols[k] = v - rows[k] * wide;
    }
    auto ask = [&](int unit0, int stage) {
        if (unit0 < 2 * p.kv_heads) {
            const int unit = unit0 + (threadIdx.x >> r.group_shift);
            const bool live = unit < 2 * p.kv_heads;
            const int kind = live && unit >= p.kv_heads ? 1 : 0, head = live ? unit - kind * p.kv_heads : 0;
            const uint32_t ld16 = kind ? r.ld16[1] : r.ld16[0];
            const uint4* src = reinterpret_cast<const uint4*>(kind ? r.in[1] : r.in[0]) +
                               (at.row * static_cast<long long>(ld16) + head * wide);
            const uint32_t to = ring + stage * S::BYTES;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k >= r.held) break;
                const bool take = live && tid + (k << r.group_shift) < count;
                kv_copy16(to + k * (THREADS * 16), src + (take ? rows[k] * ld16 + cols[k] : 0u), take);
            }
            if (at.a > 0) kv_copy4(to + S::VECTORS - threadIdx.x * 12, p.head_scale(kind, at.id, head), live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int step = r.splits * per_cta;
    int stage = 0;
#pragma unroll
    for (int k = 0; k < KV_WRITE_STAGES - 1; ++k) ask(split * per_cta + k * step, k);
    for (int unit0 = split * per_cta; unit0 < 2 * p.kv_heads; unit0 += step) {
        const int unit = unit0 + (threadIdx.x >> r.group_shift);
        const bool live = unit < 2 * p.kv_heads;
        const int kind = live && unit >= p.kv_heads ? 1 : 0, head = live ? unit - kind * p.kv_heads : 0;
        uint8_t* page = p.head_codes(kind, at.id, head);
        float* scale = p.head_scale(kind, at.id, head);
        asm volatile("cp.async.wait_group %0;" ::"n"(KV_WRITE_STAGES - 2) : "memory");
        const uint8_t* from = smem + stage * S::BYTES + threadIdx.x * 16;
        uint4 x[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k >= r.held) break;
            x[k] = *reinterpret_cast<const uint4*>(from + k * (THREADS * 16));
        }
        const float before = at.a > 0 ? *reinterpret_cast<const float*>(from + S::VECTORS - threadIdx.x * 12) : 0.0f;
        ask(unit0 + (KV_WRITE_STAGES - 1) * step, stage == 0 ? KV_WRITE_STAGES - 1 : stage - 1);
        stage = stage == KV_WRITE_STAGES - 1 ? 0 : stage + 1;
        __nv_bfloat162 m2 = __floats2bfloat162_rn(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (k >= r.held) break;
            m2 = kv_amax2(x[k].x, kv_amax2(x[k].y, kv_amax2(x[k].z, kv_amax2(x[k].w, m2))));
        }
        float m = largest(fmaxf(__low2float(m2), __high2float(m2)));
        const bool inf = m == __int_as_float(0x7f800000);
        if (__syncthreads_or(inf)) {  // seldom: the scale goes by the finite values
            float f = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                if (k >= r.held) break;
                f = kv_amax_finite(x[k].x, kv_amax_finite(x[k].y, kv_amax_finite(x[k].z, kv_amax_finite(x[k].w, f))));
            }
            m = largest(f);
        }
        int e = kv_exponent(m);
        float ratio = 1.0f;  // old codes' factor
        if (at.a > 0) {
            // The page's scale so far; one that no write can have left (not in (0, 2^120]) makes its old codes NaN.
            if (before > 0.0f && before <= kv_pow2(120)) {
                const uint32_t bits = __float_as_uint(before);
                e = max(e, static_cast<int>(bits >> 23) - 127 + ((bits & 0x7fffffu) != 0 ? 1 : 0));
                ratio = before * kv_pow2(-e);
            } else {
                ratio = __int_as_float(0x7fffffff);
            }
        }
        if (!live) continue;
        const __nv_bfloat162 inv = __float2bfloat162_rn(kv_pow2(-e));
        uint8_t* to = page + at.a * p.d + tid * 8;
        auto put = [&](auto with_inf) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (tid + (k << r.group_shift) < count)
                    *reinterpret_cast<uint2*>(to + (k << (r.group_shift + 3))) = kv_quant8<with_inf.value>(x[k], inv);
        };
        if (inf)
            put(std::true_type{});
        else
            put(std::false_type{});
        if (at.a > 0 && ratio != 1.0f) {
            uint2* old = reinterpret_cast<uint2*>(page);
            for (int v = tid; v < at.a * wide; v += group) {
                uint2 c = old[v];
                c.x = kv_requant4(c.x, ratio);
                c.y = kv_requant4(c.y, ratio);
                old[v] = c;
            }
        }
        if (tid == 0) *scale = kv_pow2(e);
    }
}

// Four codes as values, rounded to bf16.
__device__ __forceinline__ uint2 kv_values4(uint32_t c, float scale) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(c)), b = f16x2_to_float2(e4m3x2_hi_to_f16x2(c));
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * scale, a.y * scale), hi = __floats2bfloat162_rn(b.x * scale, b.y * scale);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__global__ void __launch_bounds__(KV_READ_THREADS) kv_read_kernel(const KvRows r, const KvPool p) {
    constexpr int NV = 4;
    const int group = 1 << r.group_shift, per_cta = KV_READ_THREADS >> r.group_shift;
    const int item = blockIdx.x / r.splits, split = blockIdx.x % r.splits;
    const int tid = threadIdx.x & (group - 1), wide = p.d >> 3;
    grid_dependency_wait();
    grid_launch_dependents();
    KvPage at;
    if (!kv_pick(r, p, item, at)) return;
    const int count = (at.b - at.a) * wide;
    for (int unit = split * per_cta + (threadIdx.x >> r.group_shift); unit < 2 * p.kv_heads; unit += r.splits * per_cta) {
        const int kind = unit >= p.kv_heads ? 1 : 0;
        const int head = unit - kind * p.kv_heads;
        const long long ld = kind ? r.ld[1] : r.ld[0];
        __nv_bfloat16* dst = (kind ? r.out[1] : r.out[0]) + at.row * ld + head * p.d;
        const uint2* src = reinterpret_cast<const uint2*>(p.head_codes(kind, at.id, head) + at.a * p.d);
        const float scale = *p.head_scale(kind, at.id, head);
        for (int v0 = tid; v0 < count; v0 += NV << r.group_shift) {
            uint2 c[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = v0 + (k << r.group_shift);
                if (v < count) c[k] = src[v];
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int v = v0 + (k << r.group_shift);
                if (v >= count) break;
                const uint2 lo = kv_values4(c[k].x, scale), hi = kv_values4(c[k].y, scale);
                const int row = __umulhi(v, r.per_row);
                *reinterpret_cast<uint4*>(dst + row * ld + (v - row * wide) * 8) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
        }
    }
}

// Checks that the write and the read share, then the rows' part of the launch: the pages that the call may touch.
static mp_status kv_rows_check(const void* K, const void* V, const void* kc, const void* vc, const void* ks, const void* vs,
                               const void* table, const void* cu, const void* start, bool start_needed, int nseq, int T,
                               int max_n, int kv_heads, int d, int page, int pages, int max_pages, long long ldk,
                               long long ldv, long long ld_kc, long long ld_vc, long long ld_ks, long long ld_vs,
                               const void* d_status, bool* nothing) {
    if (nseq < 0 || T < 0 || max_n < 0 || kv_heads <= 0 || d <= 0 || pages < 0 || max_pages < 0)
        return MP_ERR_INVALID_ARG;
    if (d % 16 != 0 || d > 256 || max_n > T || ldk < static_cast<long long>(kv_heads) * d ||
        ldv < static_cast<long long>(kv_heads) * d || ldk % 8 != 0 || ldv % 8 != 0 || (ldk | ldv) >> 28 != 0 ||
        !kv_pool_sizes(pages, max_pages, page, kv_heads, d, ld_kc, ld_vc, ld_ks, ld_vs))
        return MP_ERR_UNSUPPORTED_SHAPE;
    *nothing = nseq == 0 || max_n == 0;
    if (*nothing) return MP_OK;
    const mp_status st = kv_pool_pointers(kc, vc, ks, vs, table);
    if (!K || !V || !cu || (start_needed && !start)) return MP_ERR_INVALID_ARG;
    if (st != MP_OK) return st;
    auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    return aligned16(K) && aligned16(V) && word(cu) && word(start) && word(d_status) ? MP_OK : MP_ERR_MISALIGNED;
}

// The blocks of the launch, and how one finds its page and its units. A thread holds up to `most` of a unit's vectors.
static long long kv_plan(KvRows& r, const KvPool& p, int threads, int most, int blocks) {
    const long long vectors = static_cast<long long>(r.max_n < p.page ? r.max_n : p.page) * (p.d / 8);
    r.group_shift = 5;
    while ((1 << r.group_shift) < threads && vectors > static_cast<long long>(most) << r.group_shift) ++r.group_shift;
    r.per_row = static_cast<uint32_t>(((1ull << 32) + p.d / 8 - 1) / (p.d / 8));
    // A sequence's n rows touch at most this many pages, all sequences' at most `bound`.
    const long long per_seq = (static_cast<long long>(r.max_n) + p.page - 2) / p.page + 1;
    const long long bound = r.T / p.page + 2LL * r.nseq;
    const long long direct = per_seq * r.nseq;
    r.per_seq = direct <= bound ? static_cast<int>(per_seq) : 0;
    const long long pages = r.per_seq > 0 ? direct : bound;
    // Enough blocks that the last ones are a small part, each with as many units as that leaves.
    const int parts = (2 * p.kv_heads + (threads >> r.group_shift) - 1) / (threads >> r.group_shift);
    const long long splits = (blocks + pages - 1) / pages;
    r.splits = static_cast<int>(splits < parts ? splits : parts);
    return pages * r.splits;
}

static KvPool kv_pool(uint8_t* kc, uint8_t* vc, float* ks, float* vs, const int32_t* table, int pages, int max_pages,
                      int page, int kv_heads, int d, long long ld_kc, long long ld_vc, long long ld_ks, long long ld_vs) {
    KvPool p{};
    p.codes[0] = kc;
    p.codes[1] = vc;
    p.scales[0] = ks;
    p.scales[1] = vs;
    p.ld_codes[0] = ld_kc;
    p.ld_codes[1] = ld_vc;
    p.ld_scales[0] = ld_ks;
    p.ld_scales[1] = ld_vs;
    p.table = table;
    p.pages = pages;
    p.max_pages = max_pages;
    p.page = page;
    p.kv_heads = kv_heads;
    p.d = d;
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    return p;
}

}  // namespace mptp

using namespace mptp;

extern "C" mp_status mp_kv_cache_write(const mp_bf16* K, const mp_bf16* V, uint8_t* kc, uint8_t* vc, float* ks, float* vs,
                                       const int32_t* page_table, const int32_t* cu, const int32_t* start, int nseq,
                                       int T, int max_n, int kv_heads, int d, int page, int pages, int max_pages,
                                       long long ldk, long long ldv, long long ld_kc, long long ld_vc, long long ld_ks,
                                       long long ld_vs, uint32_t* d_status, void* stream) {
    bool nothing = false;
    mp_status st = kv_rows_check(K, V, kc, vc, ks, vs, page_table, cu, start, true, nseq, T, max_n, kv_heads, d, page, pages,
                                 max_pages, ldk, ldv, ld_kc, ld_vc, ld_ks, ld_vs, d_status, &nothing);
    if (st != MP_OK || nothing) return st;
    const KvPool p = kv_pool(kc, vc, ks, vs, page_table, pages, max_pages, page, kv_heads, d, ld_kc, ld_vc, ld_ks, ld_vs);
    KvRows r{};
    r.in[0] = reinterpret_cast<const __nv_bfloat16*>(K);
    r.in[1] = reinterpret_cast<const __nv_bfloat16*>(V);
    r.ld[0] = ldk;
    r.ld[1] = ldv;
    r.cu = cu;
    r.start = start;
    r.nseq = nseq;
    r.T = T;
    r.max_n = max_n;
    r.status = d_status;
    const int vectors = (max_n < page ? max_n : page) * (d / 8);  // of a unit
    const int threads = vectors > 8 * KV_WRITE_THREADS ? 2 * KV_WRITE_THREADS : KV_WRITE_THREADS;
    const long long grid = kv_plan(r, p, threads, 8, KV_WRITE_BLOCKS);
    if (grid > 0x7fffffffLL) return MP_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    st = check_device(&sms);
    if (st != MP_OK) return st;
    r.held = ceil_div(vectors, 1 << r.group_shift);
    r.ld16[0] = static_cast<uint32_t>(ldk >> 3);
    r.ld16[1] = static_cast<uint32_t>(ldv >> 3);
    auto launch = [&](auto kernel, int smem) {
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, static_cast<cudaStream_t>(stream), r, p);
    };
    constexpr int N = KV_WRITE_THREADS;
    const cudaError_t e = r.held > 8    ? launch(kv_write_kernel<16, 2 * N>, KvStage<16, 2 * N>::SMEM)
                          : threads > N ? launch(kv_write_kernel<8, 2 * N>, KvStage<8, 2 * N>::SMEM)
                          : r.held > 1  ? launch(kv_write_kernel<8, N>, KvStage<8, N>::SMEM)
                                        : launch(kv_write_kernel<1, N>, KvStage<1, N>::SMEM);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

extern "C" mp_status mp_kv_cache_read(const uint8_t* kc, const uint8_t* vc, const float* ks, const float* vs, mp_bf16* K,
                                      mp_bf16* V, const int32_t* page_table, const int32_t* cu, const int32_t* start,
                                      int nseq, int T, int max_n, int kv_heads, int d, int page, int pages, int max_pages,
                                      long long ldk, long long ldv, long long ld_kc, long long ld_vc, long long ld_ks,
                                      long long ld_vs, uint32_t* d_status, void* stream) {
    bool nothing = false;
    mp_status st = kv_rows_check(K, V, kc, vc, ks, vs, page_table, cu, start, false, nseq, T, max_n, kv_heads, d, page,
                                 pages, max_pages, ldk, ldv, ld_kc, ld_vc, ld_ks, ld_vs, d_status, &nothing);
    if (st != MP_OK || nothing) return st;
    const KvPool p = kv_pool(const_cast<uint8_t*>(kc), const_cast<uint8_t*>(vc), const_cast<float*>(ks),
                             const_cast<float*>(vs), page_table, pages, max_pages, page, kv_heads, d, ld_kc, ld_vc, ld_ks,
                             ld_vs);
    KvRows r{};
    r.out[0] = reinterpret_cast<__nv_bfloat16*>(K);
    r.out[1] = reinterpret_cast<__nv_bfloat16*>(V);
    r.ld[0] = ldk;
    r.ld[1] = ldv;
    r.cu = cu;
    r.start = start;
    r.nseq = nseq;
    r.T = T;
    r.max_n = max_n;
    r.status = d_status;
    const long long grid = kv_plan(r, p, KV_READ_THREADS, 4, KV_READ_BLOCKS);
    if (grid > 0x7fffffffLL) return MP_ERR_UNSUPPORTED_SHAPE;
    int sms = 0;
    st = check_device(&sms);
    if (st != MP_OK) return st;
    const cudaError_t e = launch_pdl(kv_read_kernel, dim3(static_cast<unsigned>(grid)), dim3(KV_READ_THREADS), 0,
                                     static_cast<cudaStream_t>(stream), r, p);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
