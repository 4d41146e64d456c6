// Entry point of the attention over the 8-bit cache: mp_attn_cache_fwd.
//
// The last nq tokens of a sequence attend to its cached keys and values as they are held, e4m3 codes with a scale for each
// page and head. A key head's rows are the nq * group queries that read it (group = heads / kv_heads):
//   S = scale * scale_k * (q . code_k),  P = exp(S - max),  O = sum P * scale_v * code_v / sum P
//
// Bound by memory with up to eight rows: every cached byte comes from memory once and meets `rows` queries, 2 * rows flops a
// byte. With more rows the warps' own instructions bound: 32 sequences of 8192 tokens and eight key heads take 91 us for 8 rows,
// 116 for 16 and 212 for 32, while two warps on each scheduler issue in half of its cycles. (A head's row tiles beyond the first
// read the cache again, from L2 where they follow soon: 32 rows took 545 MB from memory for 537 of cache.)
//
// A warp reads 32 tokens' codes into its own ring in shared memory (cp.async, 16 bytes a lane, two tiles ahead) and feeds mma.sync
// with the cache as the 16-row operand and the queries as the 8-column one:
//   S^T [keys x queries] = K Q^T in m16n8k32 of e4m3, the codes as they are: a lane's 16 bytes of a key row are its elements
//     of two products (the summed index may be taken in any order, the same for Q);
//   O^T [d x queries] += V^T P^T in m16n8k16 of halves: bytes of two key rows are interleaved into pairs of keys and turned
//     into halves (exact), P^T comes from S^T by transposing 8x8 blocks (movmatrix).
// With the queries as columns, eight rows fill a product that sixteen would share otherwise, and a column's statistics
// and its sums in O^T lie in the same lane. The tensor cores' 5th-generation products (tcgen05) would need their operands in
// shared or tensor memory, V one more trip for every cached byte, for 128 rows of which a decoded token has eight.
//
// Numbers. Q is scaled per row by a power of two into [128, 256) at its largest and split into two e4m3 pieces, q1 + q2 / 32:
// four of bf16's eight bits each, exact but for elements below 2^-13 of the largest, which keep 2^-22 of it. Both pieces have
// sums of their own (fp32, as every sum and statistic here). Each row has two references, which the largest so far passes by 8
// powers of two at most, of its scores and of its scores plus the logarithm of scale_v. Relative to the second, probabilities times
// scales, 2^7 or more at their largest, are rounded to halves: 2^-11 of a value, at least 2^-25 absolutely, 2^-32 of the largest
// P * scale_v among the tokens that the row sees, whatever scales other pages have. (With one reference for all rows of a warp's
// run, the largest scale met, pages 2^21 below it lost bits and 2^32 below it everything.) Exponentials give the roots of P
// and of a scale over its reference, which are multiplied and squared: P below 2^-126 counts where scale_v makes up for it.
//
// Work. The tiles of 32 keys of all (sequence, row tile, key head) items stand in one line, AC_ITEM places for what an item
// costs besides in front of each item's; the line is split evenly among the CTAs and a CTA's run among its warps. A warp
// walks its run alone, without a barrier: an item that lies within it is finished from registers. Runs that begin or
// end inside an item leave a record in shared memory, joined once at the CTA's end; an item that several CTAs share leaves
// a part of each in the workspace, which a second kernel adds: one block for every CTA that an item goes on from, so that
// an item's parts less one share its elements and a thread has two to five parts to add, whatever their number (20.5 us for
// one sequence of 131 k tokens, 76 parts an item, 21.2 for 77 sequences, three parts or two; a block a row 0.7 and 1.8 longer, the CTA
// that comes last adding them alone 6 and 3). A record and a part are the output of their own tiles with its sum, and a join
// weighs them by their shares of all sums: sums in units of the values would pass fp32's range where values come near bf16's.
//
// Measured: 128 sequences of 3190 to 8192 tokens, 64 heads of 128 on eight, 229 us, 6.5 TB/s, 96 % of a copy's rate; a call takes
// 11 us besides its bytes (a warp's first tile is there after 3.7, lengths, table and codes in a row; joins and their launch 4).
#include "mptp_kv_cache.cuh"
#include "mptp_launch.cuh"

namespace mptp {

constexpr int AC_WARPS = 8;
constexpr int AC_THREADS = AC_WARPS * 32;
constexpr int AC_TILE = 32;     // keys
constexpr int AC_ITEM = 4;      // places of an item besides its tiles
constexpr int AC_CTAS = 152;    // one on each SM: the workspace's parts
#define AC_NONE __int_as_float(0xff800000)  // -inf: no key seen
constexpr int AC_JOIN = 256;       // threads of a block of the join
constexpr int AC_BATCH = 3;        // parts in flight in each
constexpr int AC_SEQS = 4;         // sequences a lane looks at in one step
// In powers of four, as every score, reference and scale in logarithms here: where the largest P and the largest P * scale_v that a
// reference is made for come to lie, and how far they may come before it is made anew (2^15: halves end at 2^16).
constexpr float AC_P = 4.0f, AC_PV = 3.5f, AC_TOP = 7.5f;
constexpr float AC_FAR = -3.0e38f;   // a row that has seen no key, as its reference: no score comes so low
constexpr float AC_UNSEEN = 100.0f;  // dm of a row whose tokens so far have the value scale zero: below any other (2^-149)
constexpr float AC_LOG2E = 1.4426950408889634f;
constexpr float AC_LN2 = 0.6931471805599453f;

// An item that goes on from a CTA into the next: the CTA that began it and the number of those that share it (0: none).
struct AcItem {
    int parts, first, query, member, rows, head;  // query and member of a group of row 0
};

struct AcArgs {
    const __nv_bfloat16* Q;
    __nv_bfloat16* O;
    float* LSE;
    const int32_t* cu_q;
    const int32_t* lens;
    AcItem* items;  // [AC_CTAS]
    float* parts;   // [2 AC_CTAS][rows][d + 2]: what a CTA's tiles give by themselves, then (reference, sum) of each row
    long long ldq, ldo;
    int nseq, Tq, max_q, heads, group, causal;
    float inv_group, inv_kv;  // 1 / group, 1 / key heads
    float scale_log4;
    uint32_t* status;
};

// Shared-memory place of 16-byte chunk c of row r (of 32). The swizzles keep both reads free of bank conflicts: of K, a
// quarter warp takes four chunks of two neighbouring rows; of V, two chunks of rows two apart.
template <int D>
__device__ __forceinline__ int ac_place(int r, int c) {
    if constexpr (D == 128) return r * 128 + ((c ^ (r & 6) ^ ((r & 1) << 2)) << 4);
    if constexpr (D == 64) return (r ^ ((r >> 1) & 1)) * 64 + ((c ^ ((r >> 1) & 2)) << 4);
    return r * D + (c << 4);
}

__device__ __forceinline__ void ac_copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ac_copy16(uint32_t dst, const void* src, bool take) {  // zeros where not taken
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ac_copy4(uint32_t dst, const void* src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(take ? 4 : 0) : "memory");
}
__device__ __forceinline__ void ac_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ac_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ac_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ac_mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ac_transpose(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t ac_half2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float ac_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The root of 4^(m - top), 1 where nothing was seen in either.
__device__ __forceinline__ float ac_root(float m, float top) { return m == top ? 1.0f : ac_ex2(m - top); }
// 1 / sum; 0 where nothing was summed.
__device__ __forceinline__ float ac_inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

__device__ __forceinline__ float ac_lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int D, int NT>
struct AcShape {
    static constexpr int ROWS = 8 * NT;              // queries of a row tile
    // Tiles of a warp's ring. Heads of 128 are as fast with two as the memory gives (three: 243 us for 128 sequences of 5.8 k
    // tokens, two: 233); narrower ones, smaller tiles, want three (64: 61 against 56 us for 32 of 8192 and 8 key heads).
    static constexpr int STAGES = D == 128 ? 2 : 3;
    static constexpr int STAGE = 2 * AC_TILE * D;    // bytes of K and V
    static constexpr int RING = STAGES * STAGE;      // a warp's; then the record of the item that its run ends in
    static constexpr int HEAD = ROWS * D * 4;        // the record of the item that its run begins in
    static constexpr int WARP = RING + HEAD;
    static constexpr int SCALES = STAGES * 16;       // a warp's: two of K, two of V
    static constexpr int STATS = 2 * ROWS * 8;       // a warp's: (reference, sum) of its records' rows
    static constexpr int SMEM = AC_WARPS * (WARP + SCALES + STATS);
    static constexpr int PART = ROWS * (D + 2);      // floats of a part
    static_assert(HEAD <= RING && SMEM <= 231424, "shared memory");
};

// What a warp leaves of an item that it has not done alone: tiles [tile0, tile1) of `tiles`, first at place u0.
struct AcRecord {
    long long u0;  // -1: none
    int tile0, tile1, tiles;
    int query, member, rows, head;
};

// x / d. (x + 1/2) / d in fp32 lies nearer to its integer than to the next for x below 2^20; a division of integers takes as long
// as eight such.
__device__ __forceinline__ int ac_div(int x, int d, float inv) {
    return x < 1 << 20 ? static_cast<int>((static_cast<float>(x) + 0.5f) * inv) : x / d;
}

// Where the c-th of n equal shares of the line begins, total * c / n; the line in 32 bits where they hold it.
__device__ __forceinline__ void ac_share(long long total, int c, int n, long long& begin, long long& end) {
    long long each;
    if (total >> 32 == 0) {
        const unsigned low = static_cast<unsigned>(total);
        each = n == AC_CTAS ? low / AC_CTAS : low / static_cast<unsigned>(n);
    } else {
        each = total / n;
    }
    const int rest = static_cast<int>(total - each * n);  // rest * c < 2^15
    const float inv = 1.0f / static_cast<float>(n);
    begin = each * c + ac_div(rest * c, n, inv);
    end = each * (c + 1) + ac_div(rest * (c + 1), n, inv);
}

// The share that holds place x.
__device__ __forceinline__ int ac_owner(long long total, long long x, int n) {
    const unsigned long long y = static_cast<unsigned long long>(x + 1) * static_cast<unsigned>(n) - 1;
    return static_cast<int>(y >> 32 || total >> 32 ? y / static_cast<unsigned long long>(total)
                                                   : static_cast<unsigned>(y) / static_cast<unsigned>(total));
}

// One sequence's place in the line of tiles.
struct AcSeq {
    int q0, nq, len, tiles, items;  // tiles of one item; items = row tiles * key heads
};
template <int ROWS>
__device__ __forceinline__ AcSeq ac_seq(const AcArgs& a, const KvPool& p, int q0, int q1, int len) {
    AcSeq s{q0, q1 - q0, len, 1, 0};
    if (s.q0 < 0 || q1 < s.q0 || q1 > a.Tq || s.nq > a.max_q || s.len < 0 ||
        static_cast<long long>(s.len) > static_cast<long long>(p.max_pages) * p.page) {
        if (a.status != nullptr) atomicOr(a.status, KV_SEQ_RANGE);
        s.nq = s.len = 0;
    }
    s.tiles = max(1, (s.len + AC_TILE - 1) / AC_TILE);
    s.items = (s.nq * a.group + ROWS - 1) / ROWS * p.kv_heads;
    return s;
}
// Of sequences seq ... seq + N - 1, none behind the last: all of them asked for before the first is looked at.
template <int ROWS, int N>
__device__ __forceinline__ void ac_seqs(const AcArgs& a, const KvPool& p, int seq, AcSeq (&s)[N]) {
    int q[N + 1], len[N];
#pragma unroll
    for (int k = 0; k <= N; ++k) q[k] = seq + k <= a.nseq ? a.cu_q[seq + k] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k) len[k] = seq + k < a.nseq ? a.lens[seq + k] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = AcSeq{0, 0, 0, 1, 0};
        if (seq + k < a.nseq) s[k] = ac_seq<ROWS>(a, p, q[k], q[k + 1], len[k]);
    }
}

// Float2 index within a row of the join buffer: eight lanes that write the same j land in different banks.
__device__ __forceinline__ int ac_join(int i, int row) { return i ^ (((i >> 4) & 1) | ((row & 6))); }

// Row `col` of a row tile whose row 0 is head `member` of a group, as a query after that one's and a head of its group.
struct AcRow {
    int query, member;
};
__device__ __forceinline__ AcRow ac_row(const AcArgs& a, int query, int member, int col) {
    const int n = member + col, q = static_cast<int>((static_cast<float>(n) + 0.5f) * a.inv_group);  // n < 2^16 + 16: as ac_div
    return {query + q, n - q * a.group};
}

// The output x of row `row` of an item and its sum of probabilities: four elements at d.
__device__ __forceinline__ void ac_store(const AcArgs& a, int head, const AcRow& row, int d, int D, const float4& x, float top,
                                         float sum) {
    const int hd = head * a.group + row.member;
    const long long q = row.query;
    uint2 out = make_uint2(0, 0);  // a row that sees no key, whatever x holds
    if (sum != 0.0f) {
        const __nv_bfloat162 b0 = __floats2bfloat162_rn(x.x, x.y), b1 = __floats2bfloat162_rn(x.z, x.w);
        out = make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    }
    *reinterpret_cast<uint2*>(a.O + q * a.ldo + hd * D + d) = out;
    if (d == 0) a.LSE[static_cast<long long>(hd) * a.Tq + q] = sum == 0.0f ? AC_NONE : (2.0f * (top + AC_P) + log2f(sum * 0.00390625f)) * AC_LN2;
}

template <int D, int NT>
__global__ void __launch_bounds__(AC_THREADS, 1) attn_cache_kernel(const AcArgs a, const KvPool p) {
    using C = AcShape<D, NT>;
    constexpr int KS = D / 16;   // products along d of one score tile; also tiles of 16 rows of O^T
    constexpr int CH = D / 16;   // 16-byte chunks a key row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ AcRecord rec[2 * AC_WARPS];
    __shared__ long long sh_places[AC_WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    float* stats = reinterpret_cast<float*>(smem + AC_WARPS * (C::WARP + C::SCALES));  // [warp][2][row]{m, l}
    grid_dependency_wait();
    grid_launch_dependents();

    // The line's length, then the warp's run and the sequence that holds its first place: each warp by itself, lanes taking
    // AC_SEQS neighbouring sequences each (loads side by side, and no barrier where one step sees all of them).
    auto places = [&](const AcSeq& q) { return static_cast<long long>(q.items) * (q.tiles + AC_ITEM); };
    AcSeq held[AC_SEQS];
    long long mine = 0;  // places of the lane's sequences
    auto look_at = [&](int base) {
        mine = 0;
        ac_seqs<C::ROWS>(a, p, base + lane * AC_SEQS, held);
#pragma unroll
        for (int k = 0; k < AC_SEQS; ++k) mine += places(held[k]);
        long long upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += v;
        }
        return upto;
    };
    // More sequences than a warp looks at in one step: each takes an eighth, and the eighth that holds its first place again.
    constexpr int STEP = 32 * AC_SEQS;
    const int part = a.nseq > STEP ? (a.nseq + AC_WARPS * STEP - 1) / (AC_WARPS * STEP) * STEP : 0;
    long long upto = look_at(part * warp);
    long long total = __shfl_sync(0xffffffffu, upto, 31);
    if (part > 0) {
        for (int base = part * warp + STEP; base < min(part * (warp + 1), a.nseq); base += STEP)
            total += __shfl_sync(0xffffffffu, look_at(base), 31);
        if (lane == 0) sh_places[warp] = total;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < AC_WARPS; ++w) total += sh_places[w];
    }
    // As many CTAs as have a few places for each of their warps.
    const long long want = (total + 2 * AC_WARPS - 1) / (2 * AC_WARPS);
    const int ctas = static_cast<int>(want < static_cast<long long>(gridDim.x) ? want : static_cast<long long>(gridDim.x));
    const int cta = blockIdx.x;
    AcItem* left = a.items + cta;
    if (tid == 0) left->parts = 0;
    if (cta >= ctas) return;
    if (lane < 2) rec[2 * warp + lane].u0 = -1;
    long long cta_pos, cta_end;
    ac_share(total, cta, ctas, cta_pos, cta_end);
    long long pos = cta_pos + (cta_end - cta_pos) * warp / AC_WARPS;
    const long long end = cta_pos + (cta_end - cta_pos) * (warp + 1) / AC_WARPS;
    int seq = 0, first = 0;
    long long seq_start = 0;
    if (part > 0) {
#pragma unroll
        for (int w = 0; w < AC_WARPS - 1; ++w)
            if (pos >= seq_start + sh_places[w] && first == part * w) {
                seq_start += sh_places[w];
                first += part;
            }
        upto = look_at(first) + seq_start;
    }
    AcSeq s = held[0];
    for (int base = first; base < a.nseq;) {
        const unsigned here = __ballot_sync(0xffffffffu, pos < upto);
        if (here == 0) {  // pos lies before the line's end, so some step finds it
            seq_start = __shfl_sync(0xffffffffu, upto, 31);
            base += STEP;
            upto = look_at(base) + seq_start;
            continue;
        }
        // The lane that holds it walks its own sequences, then tells the others.
        const int who = __ffs(here) - 1;
        long long start = upto - mine;
        int k = 0;
        s = held[0];
#pragma unroll
        for (int j = 1; j < AC_SEQS; ++j)
            if (k == j - 1 && pos >= start + places(s)) {
                start += places(s);
                s = held[j];
                k = j;
            }
        seq = base + who * AC_SEQS + __shfl_sync(0xffffffffu, k, who);
        seq_start = __shfl_sync(0xffffffffu, start, who);
        s.q0 = __shfl_sync(0xffffffffu, s.q0, who);
        s.nq = __shfl_sync(0xffffffffu, s.nq, who);
        s.len = __shfl_sync(0xffffffffu, s.len, who);
        s.tiles = __shfl_sync(0xffffffffu, s.tiles, who);
        s.items = __shfl_sync(0xffffffffu, s.items, who);
        break;
    }

    uint8_t* ring = smem + warp * C::WARP;
    const uint32_t ring_u = smem_u32(ring);
    float* ring_scales = reinterpret_cast<float*>(smem + AC_WARPS * C::WARP + warp * C::SCALES);
    const uint32_t ring_scales_u = smem_u32(ring_scales);

    int last_seq = -1, local = 0, head = 0, row_tile = 0;  // of the item in hand
    while (pos < end) {
        while (seq < a.nseq && pos >= seq_start + places(s)) {
            seq_start += places(s);
            AcSeq one[1];
            ac_seqs<C::ROWS>(a, p, ++seq, one);
            s = one[0];
        }
        if (seq >= a.nseq) break;
        const int span = s.tiles + AC_ITEM;
        const long long ahead = pos - seq_start;
        int off0 = 0;
        if (seq == last_seq) {  // the item behind the last one
            ++local;
            if (++head == p.kv_heads) {
                head = 0;
                ++row_tile;
            }
        } else {
            local = ahead <= 0x7fffffff ? ac_div(static_cast<int>(ahead), span, __frcp_rn(static_cast<float>(span)))
                                        : static_cast<int>(ahead / span);
            off0 = static_cast<int>(ahead - static_cast<long long>(local) * span);
            row_tile = ac_div(local, p.kv_heads, a.inv_kv);
            head = local - row_tile * p.kv_heads;
            last_seq = seq;
        }
        const int take = static_cast<int>(min(static_cast<long long>(span - off0), end - pos));
        const int tile0 = max(off0 - AC_ITEM, 0), tile1 = off0 + take - AC_ITEM;
        pos += take;
        if (tile1 <= tile0) continue;
        const int row0 = row_tile * C::ROWS;
        const int ahead0 = ac_div(row0, a.group, a.inv_group);  // queries in front of the tile's first
        const int query0 = s.q0 + ahead0, rem0 = row0 - ahead0 * a.group;
        const int rows = min(C::ROWS, s.nq * a.group - row0);
        const int32_t* table = p.table + static_cast<long long>(seq) * p.max_pages;

        // Copies of tile k of this run into stage k % STAGES. Pages are looked up one tile earlier, the first ones at once; a
        // tile of 32 keys lies in one page, or in two of 16.
        const int tiles = tile1 - tile0;
        const uint8_t* k_codes = p.head_codes(0, 0, head) + lane * 16;
        const uint8_t* v_codes = p.head_codes(1, 0, head) + lane * 16;
        // Lanes 0 to 3 bring the scales: of keys, of values, of either half.
        const float* my_scales = p.head_scale(lane >> 1 & 1, 0, head);
        const uint32_t pitch_scales = lane & 2 ? p.pitch_scales[1] : p.pitch_scales[0];
        auto page_at = [&](const uint8_t* base, int kind, int id) {
            return base + (static_cast<uint64_t>(static_cast<uint32_t>(id)) * p.pitch16[kind] << 4);
        };
        const bool two = p.page == 16;
        auto look = [&](int k, int (&id)[2]) {
            const int key = (tile0 + k) * AC_TILE;
            id[0] = -1;
            if (key < s.len) id[0] = table[key >> p.page_shift];
            id[1] = id[0];
            if (two) id[1] = key + 16 < s.len ? table[(key >> 4) + 1] : -1;
        };
        auto issue = [&](int k, const int (&id)[2]) {
            if (k < tiles) {
                const int key0 = (tile0 + k) * AC_TILE;
                const int st = k % C::STAGES;
                const uint32_t dst = ring_u + st * C::STAGE;
                const int slot = (key0 & (p.page - 1)) * D;
                const bool inside0 = static_cast<unsigned>(id[0]) < static_cast<unsigned>(p.pages);
                const bool inside1 = static_cast<unsigned>(id[1]) < static_cast<unsigned>(p.pages);
                if (key0 + AC_TILE <= s.len && inside0 && inside1) {
                    const uint8_t* ks = page_at(k_codes, 0, id[0]) + slot;
                    const uint8_t* vs = page_at(v_codes, 1, id[0]) + slot;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 1) {
                            ks = two ? page_at(k_codes, 0, id[1]) : ks + 16 * D;
                            vs = two ? page_at(v_codes, 1, id[1]) : vs + 16 * D;
                        }
#pragma unroll
                        for (int i = 0; i < CH / 2; ++i) {  // 16 rows, 32 chunks a step
                            const int c = i * 32 + lane;
                            const uint32_t at = dst + ac_place<D>(h * 16 + c / CH, c % CH);
                            ac_copy16(at, ks + i * 512);
                            ac_copy16(at + AC_TILE * D, vs + i * 512);
                        }
                    }
                    if (lane < 4) {
                        const uint32_t page = static_cast<uint32_t>(lane & 1 ? id[1] : id[0]);
                        ac_copy4(ring_scales_u + (st * 4 + lane) * 4, my_scales + static_cast<uint64_t>(page) * pitch_scales, true);
                    }
                } else {
                    // The sequence's last tile, or a page that is not in the pool: zeros where there is no token, NaN as the
                    // scales of such a page.
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool inside = h ? inside1 : inside0;
                        const int page = inside ? id[h] : 0;
                        const uint8_t* ks = page_at(k_codes, 0, page) + (two ? 0 : slot + h * 16 * D);
                        const uint8_t* vs = page_at(v_codes, 1, page) + (two ? 0 : slot + h * 16 * D);
#pragma unroll
                        for (int i = 0; i < CH / 2; ++i) {
                            const int c = i * 32 + lane, r = h * 16 + c / CH;
                            const uint32_t at = dst + ac_place<D>(r, c % CH);
                            const bool live = inside && key0 + r < s.len;
                            ac_copy16(at, ks + i * 512, live);
                            ac_copy16(at + AC_TILE * D, vs + i * 512, live);
                        }
                        if (lane < 4 && (lane & 1) == h) {
                            if (key0 + h * 16 < s.len && !inside) {
                                ring_scales[st * 4 + lane] = __int_as_float(0x7fffffff);
                                if (a.status != nullptr) atomicOr(a.status, KV_PAGE_RANGE);
                            } else {
                                ac_copy4(ring_scales_u + (st * 4 + lane) * 4, my_scales + static_cast<uint64_t>(page) * pitch_scales, inside);
                            }
                        }
                    }
                }
            }
            ac_commit();
        };
        int ids[C::STAGES][2];
#pragma unroll
        for (int k = 0; k < C::STAGES; ++k) look(k, ids[k]);
        // Queries: lane (g, t) has row g of each eight, the elements that its bytes of a key row meet. Asked for before the
        // copies.
        constexpr int NV = D / 32;  // 16-byte vectors of a lane
        union {
            uint4 v[NV];
            uint32_t w[NV * 4];
        } x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const AcRow row = ac_row(a, query0, rem0, n * 8 + g);
            const __nv_bfloat16* src = a.Q + row.query * a.ldq + (head * a.group + row.member) * D;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                // D = 128: 16 elements of each half; else D / 4 neighbouring ones
                const int at = D == 128 ? (k >> 1) * 64 + t * 16 + (k & 1) * 8 : t * (D / 4) + k * 8;
                x[n].v[k] = make_uint4(0, 0, 0, 0);
                if (n * 8 + g < rows) x[n].v[k] = *reinterpret_cast<const uint4*>(src + at);
            }
        }
#pragma unroll
        for (int k = 0; k < C::STAGES - 1; ++k) issue(k, ids[k]);

        uint32_t qf[2][NT][KS];  // pieces q1, q2
        float fq[NT][2];         // factor from a product to a score in powers of four, for columns 2t, 2t + 1
        int limit[NT][2];        // keys that those columns see
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float m = 0.0f;
#pragma unroll
            for (int k = 0; k < NV * 4; ++k)
                m = fmaxf(m, fmaxf(fabsf(__uint_as_float(x[n].w[k] << 16)), fabsf(__uint_as_float(x[n].w[k] & 0xffff0000u))));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // An infinity in the row makes all of it NaN (e4m3 would hold it as 448).
            const float nan = m < __int_as_float(0x7f800000) ? 0.0f : __int_as_float(0x7fffffff);
            const int e = max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100) - 7;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - min(e, 120)) << 23);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t piece[2] = {0, 0};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t w = x[n].w[2 * k + j];
                    const float q0 = __uint_as_float(w << 16) * down + nan, q1 = __uint_as_float(w & 0xffff0000u) * down + nan;
                    const uint32_t c = float2_to_e4m3x2(q0, q1);
                    const float2 held = f16x2_to_float2(e4m3x2_to_f16x2(c));
                    piece[0] |= c << (16 * j);
                    piece[1] |= float2_to_e4m3x2((q0 - held.x) * 32.0f, (q1 - held.y) * 32.0f) << (16 * j);
                }
                qf[0][n][k] = piece[0];
                qf[1][n][k] = piece[1];
            }
            const float f = __uint_as_float(static_cast<uint32_t>(min(e, 120) + 127) << 23) * a.scale_log4;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fq[n][j] = __shfl_sync(0xffffffffu, f, (2 * t + j) * 4);
                const int col = n * 8 + 2 * t + j;
                limit[n][j] = col < rows && a.causal ? s.len - s.nq + ac_row(a, ahead0, rem0, col).query + 1 : s.len;
            }
        }
        // Below this tile no column is masked.
        const int clear = a.causal ? s.len - s.nq + ahead0 + 1 : s.len;

        float o[KS][NT][4];
        // P = 4^(s - m0) and its sum; o is the sum of P * scale_v * 4^dm times the values' codes.
        float m0[NT][2], l[NT][2], dm[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m0[n][0] = m0[n][1] = AC_FAR;
            dm[n][0] = dm[n][1] = AC_UNSEEN;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int j = 0; j < KS; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
        }
        int id[2] = {ids[C::STAGES - 1][0], ids[C::STAGES - 1][1]};
        for (int k = 0; k < tiles; ++k) {
            ac_wait<C::STAGES - 2>();
            __syncwarp();
            issue(k + C::STAGES - 1, id);
            look(k + C::STAGES, id);
            const int st = k % C::STAGES;
            const uint8_t* kt = ring + st * C::STAGE;
            const uint8_t* vt = kt + AC_TILE * D;
            const float* sc = ring_scales + st * 4;
            const int key0 = (tile0 + k) * AC_TILE;

            float z[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float z2[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 4; ++c) z[h][n][c] = z2[n][c] = 0.0f;
                uint32_t kw[2][KS];  // words of rows g and g + 8
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = h * 16 + r * 8 + g;
                    if constexpr (D == 96) {
#pragma unroll
                        for (int i = 0; i < 3; ++i) {
                            const uint2 v = *reinterpret_cast<const uint2*>(kt + row * D + t * 24 + i * 8);
                            kw[r][2 * i] = v.x;
                            kw[r][2 * i + 1] = v.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4*>(kt + ac_place<D>(row, i * 4 + t));
                            kw[r][4 * i] = v.x;
                            kw[r][4 * i + 1] = v.y;
                            kw[r][4 * i + 2] = v.z;
                            kw[r][4 * i + 3] = v.w;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < KS; i += 2)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        ac_mma8(z[h][n], kw[0][i], kw[1][i], kw[0][i + 1], kw[1][i + 1], qf[0][n][i], qf[0][n][i + 1]);
                        ac_mma8(z2[n], kw[0][i], kw[1][i], kw[0][i + 1], kw[1][i + 1], qf[1][n][i], qf[1][n][i + 1]);
                    }
                // Scores in powers of four; lane (g, t) has keys g, g + 8 of each 16 and queries 2t, 2t + 1 of each 8.
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // a value scale that is NaN or infinite shows in the scores, so in the rows that see them alone
                    const float ks = fmaf(sc[2 + h], 0.0f, sc[h]);
                    const float f[2] = {ks * fq[n][0], ks * fq[n][1]};
#pragma unroll
                    for (int c = 0; c < 4; ++c) z[h][n][c] = fmaf(z2[n][c], 0.03125f, z[h][n][c]) * f[c & 1];
                }
            }
            if (key0 + AC_TILE > clear) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (key0 + h * 16 + (c >> 1) * 8 + g >= limit[n][c & 1]) z[h][n][c] = AC_NONE;
            }
            const float lv[2] = {0.5f * ac_lg2(sc[2]), 0.5f * ac_lg2(sc[3])};  // the values' scales
            float high[NT][2][2];  // largest score of either half
            bool higher = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) high[n][j][h] = fmaxf(z[h][n][j], z[h][n][2 + j]);
                    const float h0 = high[n][j][0] - m0[n][j], h1 = high[n][j][1] - m0[n][j];
                    higher |= fmaxf(fmaxf(h0, h1), fmaxf(h0 + (lv[0] + dm[n][j]), h1 + (lv[1] + dm[n][j]))) > AC_TOP;
                }
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float before = m0[n][j], d0 = dm[n][j];
                        float v = fmaxf(fmaxf(high[n][j][0], high[n][j][1]), before + AC_P);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                        const float after = v > AC_FAR ? v - AC_P : AC_FAR;
                        const float down = before - after;
                        // The largest exponent of P * scale_v, that of o's reference so far among them.
                        float w = before == AC_FAR ? AC_NONE : AC_PV - d0 + down;
                        w = fmaxf(w, fmaxf(high[n][j][0] - after + lv[0], high[n][j][1] - after + lv[1]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, off));
                        m0[n][j] = after;
                        dm[n][j] = w == AC_NONE ? AC_UNSEEN : AC_PV - w;
                        l[n][j] *= ac_ex2(2.0f * down);
                        const float f = ac_ex2(2.0f * (down + (dm[n][j] - d0)));
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            o[i][n][j] *= f;
                            o[i][n][2 + j] *= f;
                        }
                    }
            }
            uint32_t pt[2][NT][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // Roots: their products hold what P and a scale far apart alone may not.
                    const float w0 = ac_ex2(fminf(lv[h] + dm[n][0], 127.0f)), w1 = ac_ex2(fminf(lv[h] + dm[n][1], 127.0f));
                    const float p0 = ac_ex2(z[h][n][0] - m0[n][0]), p1 = ac_ex2(z[h][n][1] - m0[n][1]);
                    const float p2 = ac_ex2(z[h][n][2] - m0[n][0]), p3 = ac_ex2(z[h][n][3] - m0[n][1]);
                    l[n][0] += fmaf(p0, p0, p2 * p2);
                    l[n][1] += fmaf(p1, p1, p3 * p3);
                    const float v0 = p0 * w0, v1 = p1 * w1, v2 = p2 * w0, v3 = p3 * w1;
                    pt[h][n][0] = ac_transpose(ac_half2(v0 * v0, v1 * v1));
                    pt[h][n][1] = ac_transpose(ac_half2(v2 * v2, v3 * v3));
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                constexpr int VW = D / 32;  // words of a lane in one key row
                uint32_t vw[4][VW];         // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = h * 16 + 2 * t + (r & 1) + (r >> 1) * 8;
                    if constexpr (D == 128) {
                        const uint4 v = *reinterpret_cast<const uint4*>(vt + ac_place<D>(row, g));
                        vw[r][0] = v.x;
                        vw[r][1] = v.y;
                        vw[r][2] = v.z;
                        vw[r][3] = v.w;
                    } else if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(vt + ac_place<D>(row, g >> 1) + (g & 1) * 8);
                        vw[r][0] = v.x;
                        vw[r][1] = v.y;
                    } else {
#pragma unroll
                        for (int i = 0; i < VW; ++i)
                            vw[r][i] = *reinterpret_cast<const uint32_t*>(vt + row * D + g * 12 + i * 4);
                    }
                }
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                    const uint32_t lo = __byte_perm(vw[0][j / 2], vw[1][j / 2], sel);
                    const uint32_t hi = __byte_perm(vw[2][j / 2], vw[3][j / 2], sel);
                    const uint32_t f[4] = {e4m3x2_to_f16x2(lo), e4m3x2_hi_to_f16x2(lo), e4m3x2_to_f16x2(hi),
                                           e4m3x2_hi_to_f16x2(hi)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) ac_mma(o[j][n], f, pt[h][n][0], pt[h][n][1]);
                }
            }
        }
        ac_wait<0>();
        __syncwarp();  // the ring and the scales are free

#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
        // What a row's tiles give by themselves: the sums over the probabilities' sum, in the values' units (in two steps, as the way
        // may pass what a number holds): as large as the values at most.
        float m[NT][2], to_own[NT][2], back[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[n][j] = m0[n][j] == AC_FAR ? AC_NONE : m0[n][j];
                back[n][j] = ac_ex2(-dm[n][j]);
                to_own[n][j] = back[n][j] * ac_inverse(l[n][j]);
            }
        auto own = [&](int i, int n, int c) { return o[i][n][c] * to_own[n][c & 1] * back[n][c & 1]; };
        if (tile0 == 0 && tile1 == s.tiles) {
            // The whole item: lane (g, t) has D / 8 neighbouring elements of queries 2t and 2t + 1 of each eight.
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = n * 8 + 2 * t + j;
                    if (row >= rows) continue;
                    const AcRow at = ac_row(a, query0, rem0, row);
#pragma unroll
                    for (int i = 0; i < KS; i += 2)
                        ac_store(a, head, at, g * (D / 8) + 2 * i, D,
                                 make_float4(own(i, n, j), own(i, n, 2 + j), own(i + 1, n, j), own(i + 1, n, 2 + j)), m[n][j],
                                 l[n][j]);
                }
            continue;
        }
        const int which = tile1 < s.tiles ? 1 : 0;  // the run ends in the item, or began in it
        float2* to = reinterpret_cast<float2*>(which ? ring : ring + C::RING);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = n * 8 + 2 * t + j;
                const bool none = l[n][j] == 0.0f;  // no key seen: zeros, whatever the sums hold
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    to[row * (D / 2) + ac_join(g * (D / 16) + i, row)] =
                        none ? make_float2(0.0f, 0.0f) : make_float2(own(i, n, j), own(i, n, 2 + j));
                if (g == 0)
                    *reinterpret_cast<float2*>(stats + ((warp * 2 + which) * C::ROWS + row) * 2) = make_float2(m[n][j], l[n][j]);
            }
        if (lane == 0) {
            AcRecord& r = rec[warp * 2 + which];
            r.u0 = seq_start + static_cast<long long>(local) * span;
            r.tile0 = tile0;
            r.tile1 = tile1;
            r.tiles = s.tiles;
            r.query = query0;
            r.member = rem0;
            r.rows = rows;
            r.head = head;
        }
    }
    __syncthreads();

    // Join of the records, which stand in the line's order: those of one item follow one another. First every record's share of
    // its item's sum, row by row, a thread each (by each element's thread for itself: 22.9 us, not 21.2, for 77 sequences).
    constexpr int RECS = 2 * AC_WARPS;
    __shared__ float2 shares[RECS][C::ROWS];  // as two factors: one number may not hold it where the values make up for it
    __shared__ float2 joined[RECS][C::ROWS];  // (reference, sum) of the item
    const long long my_u0 = rec[lane % RECS].u0;
    const unsigned mates = __match_any_sync(0xffffffffu, my_u0) & ((1u << RECS) - 1);
    if (tid < RECS * C::ROWS) {
        const int k = tid % RECS, row = tid / RECS;
        float2 ml[RECS];
        float top = AC_NONE, sum = 0.0f;
        float2 mine = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < RECS; ++j) {
            ml[j] = *reinterpret_cast<const float2*>(stats + (j * C::ROWS + row) * 2);
            if (mates >> j & 1) top = fmaxf(top, ml[j].x);
        }
        const float from = top == AC_NONE ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < RECS; ++j) {
            const float f = mates >> j & 1 ? ml[j].y * ac_ex2(2.0f * (ml[j].x - from)) : 0.0f;
            sum += f;
            if (j == k) mine = ml[j];
        }
        const float h = ac_ex2(mine.x - from);
        shares[k][row] = make_float2(h, mine.y * h * ac_inverse(sum));
        joined[k][row] = make_float2(top, sum);
    }
    __syncthreads();
    unsigned todo = __ballot_sync(0xffffffffu, my_u0 >= 0) & ((1u << RECS) - 1);
    while (todo != 0) {
        const int r0 = __ffs(todo) - 1;
        const unsigned chain = __shfl_sync(0xffffffffu, mates, r0);
        todo &= ~chain;
        const AcRecord r = rec[r0];
        const bool on = rec[31 - __clz(chain)].tile1 < r.tiles;  // goes on in the next CTA
        const bool whole = r.tile0 == 0 && !on;
        const bool begun = r.tile0 > 0;  // in an earlier CTA
        float* part = a.parts + static_cast<long long>(cta * 2 + (begun ? 0 : 1)) * C::PART;
        for (int i = tid; i < r.rows * (D / 4); i += AC_THREADS) {
            const int row = i / (D / 4), c = i % (D / 4) * 2;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < RECS; ++k) {
                if (!(chain >> k & 1)) continue;
                const float2 f = shares[k][row];
                const float2* from = reinterpret_cast<const float2*>(smem + (k >> 1) * C::WARP + (k & 1 ? 0 : C::RING)) + row * (D / 2);
                const float2 u = from[ac_join(c, row)], v = from[ac_join(c + 1, row)];
                x.x += u.x * f.x * f.y;
                x.y += u.y * f.x * f.y;
                x.z += v.x * f.x * f.y;
                x.w += v.y * f.x * f.y;
            }
            const float2 at = joined[r0][row];
            if (whole) {
                ac_store(a, r.head, ac_row(a, r.query, r.member, row), c * 2, D, x, at.x, at.y);
            } else {
                *reinterpret_cast<float4*>(part + row * D + c * 2) = x;
                if (c == 0) *reinterpret_cast<float2*>(part + C::ROWS * D + row * 2) = at;
            }
        }
        if (on && tid == 0) {
            left->first = ac_owner(total, r.u0 + AC_ITEM, ctas);
            left->parts = ac_owner(total, r.u0 + AC_ITEM + r.tiles - 1, ctas) - left->first + 1;
            left->query = r.query;
            left->member = r.member;
            left->rows = r.rows;
            left->head = r.head;
        }
    }
}

// Adds the parts of the item that goes on from CTA blockIdx.x of the kernel before, if there is one: of its float4 elements
// those that fall to this block, a few threads of a warp for each, every one a share of the parts.
template <int D, int NT>
__global__ void __launch_bounds__(AC_JOIN) attn_cache_join_kernel(const AcArgs a) {
    using C = AcShape<D, NT>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const AcItem it = a.items[blockIdx.x];
    if (it.parts == 0) return;
    const int all = it.rows * (D / 4), blocks = it.parts - 1;
    const int mine = ac_div(all + blocks - 1, blocks, __frcp_rn(static_cast<float>(blocks)));
    const int begin = (static_cast<int>(blockIdx.x) - it.first) * mine, end = min(begin + mine, all);
    // Elements of a warp at a time: a power of two that all warps together hold `mine` with, of 32 at most.
    const int shift = min(5, 32 - __clz((mine - 1) / (AC_JOIN / 32))), wide = 1 << shift;
    const int share = 32 >> shift, k0 = lane >> shift;
    for (int at = begin + (warp << shift); at < end; at += AC_JOIN / 32 << shift) {
        const int i = at + (lane & (wide - 1)), row = i / (D / 4), c = i % (D / 4);
        const bool live = i < end;
        float top = AC_NONE, sum = 0.0f;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k1 = k0; k1 < it.parts; k1 += share * AC_BATCH) {
            float2 ml[AC_BATCH];
            float4 v[AC_BATCH];
            float high = top;
#pragma unroll
            for (int j = 0; j < AC_BATCH; ++j) {
                const int k = k1 + j * share;
                ml[j] = make_float2(AC_NONE, 0.0f);
                v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!live || k >= it.parts) continue;
                // the first CTA began the item, the others found it begun
                const float* part = a.parts + static_cast<long long>((it.first + k) * 2 + (k == 0 ? 1 : 0)) * C::PART;
                ml[j] = *reinterpret_cast<const float2*>(part + C::ROWS * D + row * 2);
                v[j] = *reinterpret_cast<const float4*>(part + i * 4);
            }
#pragma unroll
            for (int j = 0; j < AC_BATCH; ++j) high = fmaxf(high, ml[j].x);
            // x is the output of the parts so far, each with its share of the sum, which is taken in two factors (as above).
            const float down = ac_root(top, high);
            top = high;
            sum *= down;
            float next = sum * down;
            float2 f[AC_BATCH];
#pragma unroll
            for (int j = 0; j < AC_BATCH; ++j) {
                f[j].x = ac_root(ml[j].x, top);
                f[j].y = ml[j].y * f[j].x;
                next += f[j].x * f[j].y;
            }
            const float inv = ac_inverse(next), keep = sum * inv;
            sum = next;
            x = make_float4(x.x * down * keep, x.y * down * keep, x.z * down * keep, x.w * down * keep);
#pragma unroll
            for (int j = 0; j < AC_BATCH; ++j) {
                f[j].y *= inv;
                x.x += v[j].x * f[j].x * f[j].y;
                x.y += v[j].y * f[j].x * f[j].y;
                x.z += v[j].z * f[j].x * f[j].y;
                x.w += v[j].w * f[j].x * f[j].y;
            }
        }
        // The lanes of an element: their reference and sum first, then each one's share of it.
        const float mine = top;
        for (int off = wide; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float h = ac_root(mine, top), own = sum * h;
        sum = own * h;
        for (int off = wide; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float share = own * ac_inverse(sum);
        x = make_float4(x.x * h * share, x.y * h * share, x.z * h * share, x.w * h * share);
        for (int off = wide; off < 32; off <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, off);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, off);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, off);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, off);
        }
        if (live && lane < wide)
            ac_store(a, it.head, ac_row(a, it.query, it.member, row), c * 4, D, x, top, sum);
    }
}

template <int D, int NT>
static cudaError_t launch_attn_cache(const AcArgs& a, const KvPool& p, cudaStream_t s) {
    using C = AcShape<D, NT>;
    auto kernel = attn_cache_kernel<D, NT>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    const cudaError_t f = launch_pdl(kernel, dim3(AC_CTAS), dim3(AC_THREADS), C::SMEM, s, a, p);
    if (f != cudaSuccess) return f;
    return launch_pdl(attn_cache_join_kernel<D, NT>, dim3(AC_CTAS), dim3(AC_JOIN), 0, s, a);
}

constexpr size_t AC_ITEM_BYTES = (AC_CTAS * sizeof(AcItem) + 15) / 16 * 16;

// Row tiles of eight queries where no sequence has more of a key head, else of sixteen. Those take 255 registers a thread and spill
// (heads of 128: 124 bytes stored, 184 loaded; of 96: 12 and 12), and twice the rows take 1.3 times as long (32 sequences of 8192
// tokens, eight key heads: 116 us instead of 91; heads of 64 72 instead of 52).
static int ac_rows(int max_q, int group) { return static_cast<long long>(max_q) * group <= 8 ? 8 : 16; }

}  // namespace mptp

using namespace mptp;

extern "C" size_t mp_attn_cache_workspace_bytes(int heads, int kv_heads, int d, int max_q) {
    if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || (d != 64 && d != 96 && d != 128) || max_q <= 0) return 0;
    const size_t part = static_cast<size_t>(ac_rows(max_q, heads / kv_heads)) * (d + 2) * sizeof(float);
    return AC_ITEM_BYTES + 2 * AC_CTAS * part;
}

extern "C" mp_status mp_attn_cache_fwd(const mp_bf16* Q, const uint8_t* kc, const uint8_t* vc, const float* ks,
                                       const float* vs, mp_bf16* O, float* LSE, const int32_t* page_table,
                                       const int32_t* cu_q, const int32_t* lens, void* workspace, size_t workspace_bytes,
                                       int nseq, int Tq, int max_q, int heads, int kv_heads, int d, int page, int pages,
                                       int max_pages, long long ldq, long long ldo, long long ld_kc, long long ld_vc,
                                       long long ld_ks, long long ld_vs, int causal, float scale, uint32_t* d_status,
                                       void* stream) {
    if (nseq < 0 || Tq < 0 || max_q < 0 || heads <= 0 || kv_heads <= 0 || d <= 0 || pages < 0 || max_pages < 0 ||
        !(scale > 0.0f) || !(scale <= 3.4028234663852886e38f))
        return MP_ERR_INVALID_ARG;
    const long long row = static_cast<long long>(heads) * d;
    if ((d != 64 && d != 96 && d != 128) || heads % kv_heads != 0 || heads > 65536 || row > 0x7fffffffLL || max_q > Tq || ldq < row ||
        ldo < row || ldq % 8 != 0 || ldo % 8 != 0 ||
        static_cast<long long>(max_q) * heads > 0x7fffffffLL - 64 ||
        !kv_pool_sizes(pages, max_pages, page, kv_heads, d, ld_kc, ld_vc, ld_ks, ld_vs))
        return MP_ERR_UNSUPPORTED_SHAPE;
    if (nseq == 0 || max_q == 0) return MP_OK;
    if (!Q || !O || !LSE || !cu_q || !lens) return MP_ERR_INVALID_ARG;
    mp_status st = kv_pool_pointers(kc, vc, ks, vs, page_table);
    if (st != MP_OK) return st;
    auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    if (!aligned16(Q) || !aligned16(O) || !word(LSE) || !word(cu_q) || !word(lens) || !word(d_status))
        return MP_ERR_MISALIGNED;
    if (!workspace || !aligned16(workspace) || workspace_bytes < mp_attn_cache_workspace_bytes(heads, kv_heads, d, max_q))
        return MP_ERR_WORKSPACE;
    int sms = 0;
    st = check_device(&sms);
    if (st != MP_OK) return st;

    KvPool p{};
    p.codes[0] = const_cast<uint8_t*>(kc);
    p.codes[1] = const_cast<uint8_t*>(vc);
    p.scales[0] = const_cast<float*>(ks);
    p.scales[1] = const_cast<float*>(vs);
    p.ld_codes[0] = ld_kc;
    p.ld_codes[1] = ld_vc;
    p.ld_scales[0] = ld_ks;
    p.ld_scales[1] = ld_vs;
    p.pitch16[0] = static_cast<uint32_t>(ld_kc >> 4);
    p.pitch16[1] = static_cast<uint32_t>(ld_vc >> 4);
    p.pitch_scales[0] = static_cast<uint32_t>(ld_ks);
    p.pitch_scales[1] = static_cast<uint32_t>(ld_vs);
    p.table = page_table;
    p.pages = pages;
    p.max_pages = max_pages;
    p.page = page;
    p.kv_heads = kv_heads;
    p.d = d;
    AcArgs a{};
    a.Q = reinterpret_cast<const __nv_bfloat16*>(Q);
    a.O = reinterpret_cast<__nv_bfloat16*>(O);
    a.LSE = LSE;
    a.cu_q = cu_q;
    a.lens = lens;
    a.items = static_cast<AcItem*>(workspace);
    a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + AC_ITEM_BYTES);
    a.ldq = ldq;
    a.ldo = ldo;
    a.nseq = nseq;
    a.Tq = Tq;
    a.max_q = max_q;
    a.heads = heads;
    a.group = heads / kv_heads;
    a.inv_group = 1.0f / static_cast<float>(a.group);
    a.inv_kv = 1.0f / static_cast<float>(kv_heads);
    a.causal = causal != 0;
    a.scale_log4 = scale * (0.5f * AC_LOG2E);
    p.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    a.status = d_status;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool few = ac_rows(max_q, a.group) == 8;
    cudaError_t e;
    if (d == 64)
        e = few ? launch_attn_cache<64, 1>(a, p, s) : launch_attn_cache<64, 2>(a, p, s);
    else if (d == 96)
        e = few ? launch_attn_cache<96, 1>(a, p, s) : launch_attn_cache<96, 2>(a, p, s);
    else
        e = few ? launch_attn_cache<128, 1>(a, p, s) : launch_attn_cache<128, 2>(a, p, s);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
