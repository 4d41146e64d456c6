// Entry points of the norm of queries and keys with their rotation: mp_qk_norm_rope, mp_qk_norm_rope_bwd.
//
// Per head of d elements, with r = 1 / sqrt(mean(x^2) + eps) and n = x r:
//   forward   y = R(w * n), R the rotation of mp_rope_axes (w: the queries' or the keys' weight)
//   backward  g = R^-1 dy,  dw = sum over tokens and heads of g * n,
//             dx = r (w * g - n mean(w * g * n))
// r is computed again from x, which the backward pass reads anyway: nothing is kept between the two.
//
// Bound by memory: x once in and y once out; backward x and dy in and dx out. A head lies across G = d / (2 VEC) lanes, VEC
// rotated pairs in each, or as many unrotated elements (cosine 1, sine 0), so that the sums of squares are a few shuffles
// within the G lanes. A warp walks tokens (or a share of a token's steps where tokens are few), as many heads at once as it has
// lanes for; the angles' sines are computed once a token, and with the weight they make two coefficients an element, y = r (x P +
// partner Q). All of it is fp32, two elements an instruction, and each output is rounded once.
// A lane keeps to query heads or to key heads. Where lanes for both kinds side by side take no more steps than warps for
// either kind alone (16 and 4 heads of 96, five at once: four steps, not four and one), a warp has both (16,384 tokens of those
// 22.6 us forward and 38.4 backward, apart 27.7 and 41.0; 1111 tokens of 16 and 16 heads of 64 3.3 and 8.0, apart 4.2 and 9.7).
// 28,350 tokens of 36 heads of 128: 82 us, 6.4 TB/s, 94 % of a copy's rate.
// The weights' gradients: a lane of the backward pass keeps its columns' sums in registers over all its tokens, a block
// adds its lanes' in shared memory and writes two rows of the workspace, a second kernel adds the rows: fixed order, no
// atomics.
#include "mptp_internal.h"
#include "mptp_launch.cuh"
#include "mptp_ptx.cuh"
#include "mptp_rope.cuh"

namespace mptp {

constexpr int QKN_WARPS = 4;         // warps of a block
constexpr int QKN_STAGES = 4;        // steps in flight, and the one in hand
constexpr int QKN_RUN = 48;          // steps of a warp of the forward pass
// Of 32 lanes' squares of a head, none larger than this, the sum lies within fp32's range. (The test comes before the lanes' sum: behind
// it, where it could wait for the exchanges, 8192 tokens of 20 heads of 72 take 15.5 us forward, not 15.0.)
constexpr float QKN_MOST = 4.0e36f;
// Blocks on an SM, as many as registers allow without spills: narrow lanes (VEC 4) one more (8192 tokens of 20 heads of 72 16.5 us
// forward with five, 19.6 with four, 18.3 with six; backward 24.4 with four, 25.5 with three, 26.7 with five).
constexpr int qkn_per_sm(bool wide, bool backward) { return wide ? (backward ? 3 : 4) : backward ? 4 : 5; }
constexpr int QKN_BWD_ROWS = 4 * 152;  // pairs of rows of the workspace at most: blocks of the backward pass

struct QkNormArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* dy;
    __nv_bfloat16* y;  // backward: dx
    const __nv_bfloat16* wq;
    const __nv_bfloat16* wk;
    const int32_t* pos;  // [axes][T]
    float* sums;         // [blocks][2][d]
    long long ldx, ldy, lddy;
    int T, heads, q_heads, d, pairs, axes;
    // Of warps that have query heads, or both kinds, and of those of the blocks from q_blocks on, key heads alone:
    int shares, k_shares;  // log2 of the warps that share a token's steps
    int q_slots;           // heads at once that are queries', of the first
    int q_own, k_own;      // heads of the first lanes of either kind
    int steps, k_steps;    // of a token
    int q_blocks;
    float eps, inv_d;
};

// Where a lane's two vectors of VEC elements lie within a head.
template <int VEC, bool INTER>
struct QkLane {
    int groups, per_warp, g, sub, o0, o1;
    bool live, turns;
    __device__ __forceinline__ QkLane(int d, int pairs, int lane) {
        groups = d / (2 * VEC);
        per_warp = 32 / groups;
        g = lane % groups;
        sub = lane / groups;
        live = sub < per_warp;
        const int rotated = pairs / VEC;
        turns = g < rotated;
        o0 = INTER || !turns ? 2 * VEC * g : VEC * g;
        o1 = INTER || !turns ? o0 + VEC : o0 + pairs;
    }
};

// How the sum over a head's lanes is taken: G a power of two, three times one, or any other.
enum { QK_POW2, QK_THREE, QK_ANY };

// Sum over the G lanes of a head, in all of them; every lane of the warp takes part. Heads begin at multiples of G, so
// exchanges within a power of two that divides G stay in the head; for three times one, the other two thirds lie G / 3 and
// 2 G / 3 lanes further round the head (turn[0], turn[1]).
template <int SUM, int N>
__device__ __forceinline__ void qk_head_sum(float (&v)[N], int groups, int g, int lane, const int (&turn)[2]) {
    const int pow2 = SUM == QK_THREE ? groups / 3 : groups;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        if (off >= pow2) break;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if constexpr (SUM != QK_ANY) {
                v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
            } else {
                const float o = __shfl_down_sync(0xffffffffu, v[k], off);
                if (g + off < groups) v[k] += o;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (SUM == QK_THREE)
            v[k] += __shfl_sync(0xffffffffu, v[k], turn[0]) + __shfl_sync(0xffffffffu, v[k], turn[1]);
        if constexpr (SUM == QK_ANY) v[k] = __shfl_sync(0xffffffffu, v[k], lane - g);
    }
}

// A lane's 2 VEC elements of one head as loaded: VEC words, the first vector's, then the second's.
template <int VEC>
union QkRaw {
    typename RopeVec<VEC>::T v[2];
    uint32_t w[VEC];
};
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_load(QkRaw<VEC>& x, const __nv_bfloat16* head, const QkLane<VEC, INTER>& L) {
    using V = typename RopeVec<VEC>::T;
    x.v[0] = *reinterpret_cast<const V*>(head + L.o0);
    x.v[1] = *reinterpret_cast<const V*>(head + L.o1);
}
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_store(const float2 (&f)[VEC], __nv_bfloat16* head, const QkLane<VEC, INTER>& L) {
    using V = typename RopeVec<VEC>::T;
    QkRaw<VEC> x;
#pragma unroll
    for (int k = 0; k < VEC; ++k) x.w[k] = rope_pack(f[k].x, f[k].y);
    *reinterpret_cast<V*>(head + L.o0) = x.v[0];
    *reinterpret_cast<V*>(head + L.o1) = x.v[1];
}
template <int VEC>
__device__ __forceinline__ void qk_floats(const QkRaw<VEC>& x, float2 (&f)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) f[k] = make_float2(rope_lo(x.w[k]), rope_hi(x.w[k]));
}

// f[k] P[k] + partner Q[k]: an element's partner is the other one of its pair.
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_turn(const float2 (&f)[VEC], const float2 (&P)[VEC], const float2 (&Q)[VEC],
                                        float2 (&out)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const float2 partner = INTER ? make_float2(f[k].y, f[k].x) : f[(k + VEC / 2) % VEC];
        out[k] = fma2(f[k], P[k], mul2(partner, Q[k]));
    }
}

// The angles of a token's pairs: each lane of the warp takes every 32nd pair (a head's lanes hold the same pairs as the next
// head's, so a lane's own eight would be computed several times over) and leaves cosine and sine in the warp's `cs`.
// `table`: {turns' halves, axis} of each pair, in shared memory; `pos`: the token's positions by axis, there too. BACK: of the
// rotation back. sin.approx and cos.approx stay within 2^-20 on [-pi, pi], far below a bf16 step.
template <bool BACK>
__device__ __forceinline__ void qk_angles(const uint4* table, const int* pos, float* cs, int pairs, int lane) {
    for (int i = lane; i < pairs; i += 32) {
        const uint4 f = table[i];
        const uint32_t p = static_cast<uint32_t>(pos[f.z]);
        // the upper 32 bits of p times the 64-bit turns, a signed fraction of a turn in [-1/2, 1/2), times 2 pi / 2^32
        const uint32_t top = p * f.y + __umulhi(p, f.x) - (static_cast<int32_t>(p) < 0 ? f.x : 0u);
        const float angle = static_cast<float>(static_cast<int32_t>(top)) * (BACK ? -1.4629180792671596e-9f : 1.4629180792671596e-9f);
        float s, c;
        asm("sin.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(angle));
        asm("cos.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(angle));
        cs[i] = c;
        cs[ROPE_MAX_PAIRS + i] = s;
    }
}

// Those of a lane's pairs; cosine 1 and sine 0 where it has none.
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_take_angles(const float* cs, const QkLane<VEC, INTER>& L, float (&c)[VEC], float (&s)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; j += 4) {
        float4 u = make_float4(1.0f, 1.0f, 1.0f, 1.0f), v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (L.turns) {
            u = *reinterpret_cast<const float4*>(cs + L.g * VEC + j);
            v = *reinterpret_cast<const float4*>(cs + ROPE_MAX_PAIRS + L.g * VEC + j);
        }
        c[j] = u.x, c[j + 1] = u.y, c[j + 2] = u.z, c[j + 3] = u.w;
        s[j] = v.x, s[j + 1] = v.y, s[j + 2] = v.z, s[j + 3] = v.w;
    }
}

// Coefficients of qk_turn for elements weighted by w (null: by one).
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_coefficients(const float (&c)[VEC], const float (&s)[VEC], const float2* w,
                                                float2 (&P)[VEC], float2 (&Q)[VEC]) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        if constexpr (INTER) {
            P[k] = make_float2(c[k], c[k]);
            Q[k] = make_float2(-s[k], s[k]);
        } else {
            const int j = 2 * k % VEC;
            P[k] = make_float2(c[j], c[j + 1]);
            Q[k] = k < VEC / 2 ? make_float2(-s[j], -s[j + 1]) : make_float2(s[j], s[j + 1]);
        }
        if (w != nullptr) {
            P[k] = mul2(P[k], w[k]);
            Q[k] = mul2(Q[k], INTER ? make_float2(w[k].y, w[k].x) : w[(k + VEC / 2) % VEC]);
        }
    }
}

// A lane's elements of a weight.
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_weight(const __nv_bfloat16* w, const QkLane<VEC, INTER>& L, float2 (&f)[VEC]) {
    QkRaw<VEC> x;
    qk_load(x, w, L);
    qk_floats(x, f);
}

// `take` bytes from src, zeros behind them.
template <int BYTES>
__device__ __forceinline__ void qk_copy(uint32_t dst, const void* src, int take) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(take) : "memory");
}

// The walk of a warp: items (a token's steps, or every 2^shares-th of them) `stride` apart; in step k each G lanes take the k-th of
// their heads, `hop` elements apart. A step's loads go to the lane's own places in shared memory (cp.async: nothing of them waits in
// registers, and no lane reads another's), QKN_STAGES - 1 steps ahead; N arrays are read, and the token's positions with its
// first step. Lanes without a head get zeros.
template <int VEC, int N>
struct QkWalk {
    static constexpr int BYTES = 2 * VEC;                      // of a vector
    static constexpr int STAGE = N * 2 * BYTES * 32 + 16;      // of a warp's stage: the vectors, then the positions
    const __nv_bfloat16* src[N];   // the lane's first vector of its first head, of token 0
    const __nv_bfloat16* at[N];    // and of the step to be asked for
    long long ld[N];
    const int32_t* pos;            // lane k < axes: of axis k
    uint32_t ring, pos_ring;       // the lane's places in the first stage
    bool has_axis;
    unsigned items, stride, next;
    int shares, steps, own, hop, second, next_k, stage;  // own: the lane's heads

    __device__ __forceinline__ int first_step(unsigned item) const { return static_cast<int>(item & ((1u << shares) - 1)); }
    __device__ __forceinline__ void start() {
        next_k = first_step(next);
#pragma unroll
        for (int n = 0; n < N; ++n) at[n] = src[n] + (next >> shares) * ld[n] + next_k * hop;
    }
    __device__ __forceinline__ void fetch() {
        if (next < items) {
            const int take = next_k < own ? BYTES : 0;
            const uint32_t to = ring + stage * STAGE;
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const __nv_bfloat16* from = take != 0 ? at[n] : src[n];  // an address in the tensor either way
                qk_copy<BYTES>(to + (2 * n) * BYTES * 32, from, take);
                qk_copy<BYTES>(to + (2 * n + 1) * BYTES * 32, from + second, take);
                at[n] += hop << shares;
            }
            if (has_axis && next_k >> shares == 0) qk_copy<4>(pos_ring + stage * STAGE, pos + (next >> shares), 4);
            next_k += 1 << shares;
            if (next_k >= steps) {
                next += stride;
                start();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        stage = stage == QKN_STAGES - 1 ? 0 : stage + 1;
    }
};

template <int VEC>
__device__ __forceinline__ void qk_take(const uint8_t* at, float2 (&f)[VEC]) {
    using V = typename RopeVec<VEC>::T;
    QkRaw<VEC> x;
    x.v[0] = *reinterpret_cast<const V*>(at);
    x.v[1] = *reinterpret_cast<const V*>(at + 2 * VEC * 32);
    qk_floats(x, f);
}

// Of a head whose squares may pass fp32's range (by its width, a root mean square from 2^57 to 2^61 on): its elements times 2^-80,
// whose squares it holds, and those that count stay normal. Returns the factor, 1 for other heads.
template <int VEC>
__device__ __forceinline__ float qk_scale_down(float2 (&x)[VEC], float sum) {
    const float down = sum > QKN_MOST ? 8.271806125530277e-25f : 1.0f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = mul2(x[j], make_float2(down, down));
    return down;
}

template <int VEC, bool INTER, int SUM, bool BACKWARD>
__global__ void __launch_bounds__(QKN_WARPS * 32, qkn_per_sm(VEC == 8, BACKWARD)) qk_norm_kernel(
    const __grid_constant__ RopeTable tab, const QkNormArgs a) {
    using Walk = QkWalk<VEC, BACKWARD ? 2 : 1>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const QkLane<VEC, INTER> L(a.d, a.pairs, lane);
    // The lane's heads: every slots-th of its kind, `own` of them from head0 on.
    const bool second = static_cast<int>(blockIdx.x) >= a.q_blocks;  // keys alone
    const int q_slots = second ? 0 : a.q_slots;
    const bool keys = L.sub >= q_slots;
    const int slots = keys ? L.per_warp - q_slots : q_slots, first = keys ? a.q_heads + L.sub - q_slots : L.sub;
    const int most = keys ? a.k_own : a.q_own;
    const int own = L.live ? most - (first + (most - 1) * slots >= (keys ? a.heads : a.q_heads) ? 1 : 0) : 0;
    const int head0 = own > 0 ? first : 0;
    uint4* table = reinterpret_cast<uint4*>(smem + QKN_WARPS * QKN_STAGES * Walk::STAGE);
    float* cs = reinterpret_cast<float*>(table + ROPE_MAX_PAIRS) + warp * 2 * ROPE_MAX_PAIRS;
    for (int i = threadIdx.x; i < a.pairs; i += QKN_WARPS * 32)
        table[i] = make_uint4(static_cast<uint32_t>(tab.turns[i]), static_cast<uint32_t>(tab.turns[i] >> 32), tab.axis[i], 0);
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    const uint8_t* ring = smem + warp * QKN_STAGES * Walk::STAGE + lane * Walk::BYTES;
    Walk walk;
    walk.src[0] = a.x + head0 * a.d + L.o0;
    walk.ld[0] = a.ldx;
    if constexpr (BACKWARD) {
        walk.src[1] = a.dy + head0 * a.d + L.o0;
        walk.ld[1] = a.lddy;
    }
    walk.has_axis = lane < a.axes;
    walk.pos = a.pos + static_cast<long long>(walk.has_axis ? lane : 0) * a.T;
    walk.ring = smem_u32(ring);
    const uint8_t* pos_ring = smem + warp * QKN_STAGES * Walk::STAGE + Walk::STAGE - 16;
    walk.pos_ring = smem_u32(pos_ring) + (lane & 3) * 4;
    walk.shares = second ? a.k_shares : a.shares;
    walk.items = static_cast<unsigned>(a.T) << walk.shares;
    walk.stride = (second ? gridDim.x - a.q_blocks : a.q_blocks) * QKN_WARPS;
    walk.steps = second ? a.k_steps : a.steps;
    walk.own = own;
    walk.hop = slots * a.d;
    walk.second = L.o1 - L.o0;
    walk.stage = 0;
    unsigned item = (second ? blockIdx.x - a.q_blocks : blockIdx.x) * QKN_WARPS + warp;
    walk.next = item;
    walk.start();
#pragma unroll
    for (int k = 0; k < QKN_STAGES - 1; ++k) walk.fetch();

    const __nv_bfloat16* weight = (own > 0 ? keys : a.q_heads == 0) ? a.wk : a.wq;
    float2 w[VEC], acc[VEC], P[VEC], Q[VEC];
    if constexpr (BACKWARD) qk_weight(weight, L, w);
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = make_float2(0.0f, 0.0f);
    const int turn[2] = {lane - L.g + (L.g + L.groups / 3) % L.groups, lane - L.g + (L.g + L.groups / 3 * 2) % L.groups};
    int step = walk.first_step(item), stage = 0;
    bool fresh = true;  // a token's first step
    __nv_bfloat16* out = nullptr;
    while (item < walk.items) {
        asm volatile("cp.async.wait_group %0;" ::"n"(QKN_STAGES - 2) : "memory");
        const uint8_t* at = ring + stage * Walk::STAGE;
        if (fresh) {
            const int token = static_cast<int>(item >> walk.shares);
            float c[VEC], s[VEC];
            __syncwarp();  // the positions are there, and every lane has taken the last token's angles
            qk_angles<BACKWARD>(table, reinterpret_cast<const int*>(pos_ring + stage * Walk::STAGE), cs, a.pairs, lane);
            __syncwarp();
            qk_take_angles(cs, L, c, s);
            if constexpr (!BACKWARD) qk_weight(weight, L, w);  // again for each token: sixteen registers less
            qk_coefficients<VEC, INTER>(c, s, BACKWARD ? nullptr : w, P, Q);
            out = a.y + token * a.ldy + head0 * a.d + step * walk.hop;
            fresh = false;
        }
        float2 x[VEC], y[VEC];
        qk_take<VEC>(at, x);
        float down = 1.0f, eps = a.eps;  // x stands for x / down
        if constexpr (!BACKWARD) {
            float sum[1];
            auto squares = [&] {
                float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) ss = fma2(x[j], x[j], ss);
                sum[0] = ss.x + ss.y;
            };
            squares();
            if (__any_sync(0xffffffffu, sum[0] > QKN_MOST)) {
                float all[1] = {sum[0]};
                qk_head_sum<SUM>(all, L.groups, L.g, lane, turn);
                down = qk_scale_down(x, all[0]);
                eps = eps * down * down;
                squares();
            }
            qk_head_sum<SUM>(sum, L.groups, L.g, lane, turn);
            walk.fetch();
            const float r = rsqrtf(sum[0] * a.inv_d + eps);
            qk_turn<VEC, INTER>(x, P, Q, y);
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[j] = mul2(y[j], make_float2(r, r));
        } else {
            float2 g[VEC];
            qk_take<VEC>(at + 4 * VEC * 32, y);
            qk_turn<VEC, INTER>(y, P, Q, g);
            float sum[2];  // x^2, w g x
            auto products = [&] {
                float2 ss = make_float2(0.0f, 0.0f), dot = ss;
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    ss = fma2(x[j], x[j], ss);
                    y[j] = mul2(g[j], x[j]);
                    dot = fma2(y[j], w[j], dot);
                }
                sum[0] = ss.x + ss.y;
                sum[1] = dot.x + dot.y;
            };
            products();
            if (__any_sync(0xffffffffu, sum[0] > QKN_MOST)) {
                float all[1] = {sum[0]};
                qk_head_sum<SUM>(all, L.groups, L.g, lane, turn);
                down = qk_scale_down(x, all[0]);
                eps = eps * down * down;
                products();
            }
            qk_head_sum<SUM>(sum, L.groups, L.g, lane, turn);
            walk.fetch();
            const float r = rsqrtf(sum[0] * a.inv_d + eps);
            const float m = -(sum[1] * a.inv_d * r) * r;  // -r mean(w g n)
            const float out_r = r * down;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                acc[j] = fma2(y[j], make_float2(r, r), acc[j]);
                y[j] = mul2(fma2(x[j], make_float2(m, m), mul2(w[j], g[j])), make_float2(out_r, out_r));
            }
        }
        if (step < own) qk_store(y, out, L);
        out += walk.hop << walk.shares;
        stage = stage == QKN_STAGES - 1 ? 0 : stage + 1;
        step += 1 << walk.shares;
        if (step >= walk.steps) {
            item += walk.stride;
            step = walk.first_step(item);
            fresh = true;
        }
    }
    if constexpr (BACKWARD) {
        // Sums of the block's lanes: rows [warp, sub][d], where the rings were.
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float* red = reinterpret_cast<float*>(smem);
        if (L.live) {
            float* row = red + (warp * L.per_warp + L.sub) * a.d;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const int o = k < VEC / 2 ? L.o0 + 2 * k : L.o1 + 2 * k - VEC;
                row[o] = acc[k].x;
                row[o + 1] = acc[k].y;
            }
        }
        __syncthreads();
        // Queries' columns, then keys'; of warps with one kind that kind's.
        const int from = q_slots == 0 ? a.d : 0, to = q_slots == L.per_warp ? a.d : 2 * a.d;
        for (int i = from + threadIdx.x; i < to; i += QKN_WARPS * 32) {
            const bool k = i >= a.d;
            const float* col = red + (k ? q_slots * a.d + i - a.d : i);
            float t = 0.0f;
            for (int u = k ? L.per_warp - q_slots : q_slots; u > 0; --u, col += a.d)
#pragma unroll
                for (int v = 0; v < QKN_WARPS; ++v) t += col[v * L.per_warp * a.d];
            a.sums[static_cast<long long>(blockIdx.x) * 2 * a.d + i] = t;
        }
    }
}

// dwq and dwk from the blocks' rows [2][d], queries' in the first q_rows and keys' from k_row on: a block takes 32 of d columns
// of one of the two, 32 warps a share of the rows each.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float* sums, float* dwq, float* dwk, int q_rows, int k_row,
                                                         int rows, int d) {
    __shared__ float red[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int half = gridDim.x / 2;
    const bool keys = static_cast<int>(blockIdx.x) >= half;
    const int col = (blockIdx.x - (keys ? half : 0)) * 32 + lane;
    grid_dependency_wait();
    grid_launch_dependents();
    const float* at = sums + (keys ? d : 0) + col;
    float t = 0.0f;
    if (col < d)
#pragma unroll 8
        for (int r = (keys ? k_row : 0) + warp; r < (keys ? rows : q_rows); r += 32) t += at[static_cast<long long>(r) * 2 * d];
    red[warp][lane] = t;
    __syncthreads();
    float* out = keys ? dwk : dwq;
    if (warp != 0 || col >= d || out == nullptr) return;
#pragma unroll
    for (int k = 1; k < 32; ++k) t += red[k][lane];
    out[col] = t;
}

// The lanes' vectors are 16 bytes where each half of a head and what is not rotated divide into them, else 8.
static bool qk_wide(int d, long long pairs) { return d % 16 == 0 && pairs % 8 == 0; }

static int qk_steps(int heads, int slots) { return (heads + slots - 1) / slots; }

// How heads are dealt to lanes, warps and blocks. A warp has both kinds of heads where that takes no more steps than warps for
// either. A token's steps are shared while there would be fewer than four warps on each of 152 SMs (eight: backward of 1111
// tokens of 32 heads of 72 8.3 us instead of 7.8, forward of 300 of 40 of 128 3.9 instead of 2.8, but of 700 4.2 instead of 5.0).
// Forward: a warp walks about QKN_RUN steps, so that the blocks that end late are small. Backward: as many blocks as the chip
// holds at most (each leaves a row of sums of either kind), divided so that neither kind's last warp ends much later than the
// other's; a token's angles cost about a quarter of a step.
// Steps of a warp: 48 or no limit 29.6 us for 16,384 tokens of 20 heads of 128, 24 31.0; for 28,350 of 36 heads 48 81 us, no
// limit 82.9.
static int qk_blocks(QkNormArgs& a, bool wide, bool backward) {
    const int full = qkn_per_sm(wide, backward) * 152;  // blocks that the chip holds
    const int in_hand = 32 / (a.d / (wide ? 16 : 8)), n[2] = {a.q_heads, a.heads - a.q_heads};
    int steps[2] = {qk_steps(n[0], in_hand), qk_steps(n[1], in_hand)};
    a.q_slots = n[0] > 0 ? in_hand : 0;
    a.q_own = steps[0];
    a.k_own = steps[1];
    if (n[0] == 0) {
        steps[0] = steps[1];
        steps[1] = 0;
    } else if (n[1] > 0) {
        int both = steps[0] + steps[1] + 1, slots = 0;
        for (int q = 1; q < in_hand; ++q) {
            const int x = qk_steps(n[0], q), y = qk_steps(n[1], in_hand - q);
            if ((x > y ? x : y) < both) {
                both = x > y ? x : y;
                slots = q;
            }
        }
        if (slots > 0) {
            a.q_slots = slots;
            a.q_own = qk_steps(n[0], slots);
            a.k_own = qk_steps(n[1], in_hand - slots);
            steps[0] = both;
            steps[1] = 0;
        }
    }
    a.steps = steps[0];
    a.k_steps = steps[1];
    long long items[2], most[2], cost[2];
    int blocks[2];
    for (int i = 0; i < 2; ++i) {
        int& shares = i == 0 ? a.shares : a.k_shares;
        shares = 0;
        while ((static_cast<long long>(a.T) << shares) < 4LL * 152 && 1 << shares < steps[i]) ++shares;
        items[i] = steps[i] == 0 ? 0 : static_cast<long long>(a.T) << shares;
        const int each = (steps[i] + (1 << shares) - 1) >> shares;  // steps of an item
        cost[i] = 1 + 4 * each;
        const int run = each == 0 || each > QKN_RUN ? 1 : QKN_RUN / each;
        most[i] = (items[i] + QKN_WARPS - 1) / QKN_WARPS;
        blocks[i] = static_cast<int>(backward ? most[i] : (items[i] + run * QKN_WARPS - 1) / (run * QKN_WARPS));
        if (!backward && blocks[i] < full) blocks[i] = static_cast<int>(most[i] < full ? most[i] : full);
    }
    const int all = blocks[0] + blocks[1];
    if (!backward && all > full && blocks[0] < most[0]) {
        // Whole rounds of the chip, where warps walk several items (683 blocks, where 608 fit, took 28.9 us for what 608 do in
        // 22.6; with an item a warp 5.2 us for 700 tokens, as they come 4.3).
        const double by = static_cast<double>((all + full / 2) / full) * full / all;
        for (int i = 0; i < 2; ++i) {
            const long long b = static_cast<long long>(blocks[i] * by + 0.5);
            if (blocks[i] > 0) blocks[i] = static_cast<int>(b < 1 ? 1 : b < most[i] ? b : most[i]);
        }
    }
    if (backward && most[0] + most[1] > full) {
        if (items[1] == 0) {
            // no more than what gives every warp as many items
            const long long rounds = (most[0] + full - 1) / full;
            blocks[0] = static_cast<int>((most[0] + rounds - 1) / rounds);
        } else {
            auto rounds = [&](int i, int b) { return (items[i] + b * QKN_WARPS - 1) / (b * QKN_WARPS) * cost[i]; };
            const double share = static_cast<double>(items[0] * cost[0]) / (items[0] * cost[0] + items[1] * cost[1]);
            const int guess = static_cast<int>(full * share);
            int best = guess < 1 ? 1 : guess > full - 1 ? full - 1 : guess;
            long long span = -1;
            for (int b = guess - 8 > 1 ? guess - 8 : 1; b <= guess + 8 && b < full; ++b) {
                const long long q = rounds(0, b), k = rounds(1, full - b), t = q > k ? q : k;
                if (span < 0 || t < span) {
                    span = t;
                    best = b;
                }
            }
            blocks[0] = best;
            blocks[1] = full - best;
        }
    }
    a.q_blocks = blocks[0];
    return blocks[0] + blocks[1];
}

template <int VEC, bool INTER, int SUM, bool BACKWARD>
static cudaError_t qk_launch(const RopeTable& tab, const QkNormArgs& a, int blocks, cudaStream_t s) {
    constexpr int ring = QKN_WARPS * QKN_STAGES * QkWalk<VEC, BACKWARD ? 2 : 1>::STAGE + ROPE_MAX_PAIRS * (16 + QKN_WARPS * 8);
    constexpr int red = BACKWARD ? QKN_WARPS * 32 * 2 * VEC * 4 : 0;
    constexpr int bytes = ring > red ? ring : red;
    static_assert(bytes <= 48 * 1024, "shared memory");
    return launch_pdl(qk_norm_kernel<VEC, INTER, SUM, BACKWARD>, dim3(static_cast<unsigned>(blocks)), dim3(QKN_WARPS * 32),
                      bytes, s, tab, a);
}

template <int SUM, bool BACKWARD>
static cudaError_t qk_launch_as(const RopeTable& tab, const QkNormArgs& a, bool wide, bool inter, int blocks, cudaStream_t s) {
    if (wide) return (inter ? qk_launch<8, true, SUM, BACKWARD> : qk_launch<8, false, SUM, BACKWARD>)(tab, a, blocks, s);
    return (inter ? qk_launch<4, true, SUM, BACKWARD> : qk_launch<4, false, SUM, BACKWARD>)(tab, a, blocks, s);
}

template <bool BACKWARD>
static cudaError_t qk_dispatch(const RopeTable& tab, const QkNormArgs& a, bool wide, bool inter, int blocks, cudaStream_t s) {
    const int groups = a.d / (wide ? 16 : 8), third = groups / 3;
    if ((groups & (groups - 1)) == 0) return qk_launch_as<QK_POW2, BACKWARD>(tab, a, wide, inter, blocks, s);
    if (groups % 3 == 0 && (third & (third - 1)) == 0)
        return qk_launch_as<QK_THREE, BACKWARD>(tab, a, wide, inter, blocks, s);
    return qk_launch_as<QK_ANY, BACKWARD>(tab, a, wide, inter, blocks, s);
}

static mp_status qk_check(int T, int heads, int q_heads, int d, int axes, const int* sections, double base, float eps,
                          uint32_t flags, long long* pairs) {
    if (T < 0 || heads <= 0 || q_heads < 0 || q_heads > heads || d <= 0 || !(eps > 0.0f) || !std::isfinite(eps) ||
        !rope_valid(axes, sections, base, flags, MP_ROPE_INTERLEAVED | MP_ROPE_PER_AXIS, pairs))
        return MP_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 2 * ROPE_MAX_PAIRS || *pairs < 4 || *pairs % 4 != 0 || 2 * *pairs > d ||
        static_cast<long long>(heads) * d > 0x7fffffffLL)
        return MP_ERR_UNSUPPORTED_SHAPE;
    return MP_OK;
}

static bool qk_pitch(long long ld, int heads, int d) { return ld >= static_cast<long long>(heads) * d && ld % 8 == 0; }

static QkNormArgs qk_args(int T, int heads, int q_heads, int d, int axes, long long pairs, float eps) {
    QkNormArgs a{};
    a.T = T;
    a.heads = heads;
    a.q_heads = q_heads;
    a.d = d;
    a.pairs = static_cast<int>(pairs);
    a.axes = axes;
    a.eps = eps;
    a.inv_d = 1.0f / static_cast<float>(d);
    return a;
}

}  // namespace mptp

using namespace mptp;

extern "C" mp_status mp_qk_norm_rope(const mp_bf16* x, mp_bf16* y, const mp_bf16* wq, const mp_bf16* wk,
                                     const int32_t* pos, int T, int heads, int q_heads, int d, long long ldx,
                                     long long ldy, int axes, const int* sections, double base, float eps,
                                     uint32_t flags, void* stream) {
    long long pairs = 0;
    mp_status st = qk_check(T, heads, q_heads, d, axes, sections, base, eps, flags, &pairs);
    if (st != MP_OK) return st;
    if (!qk_pitch(ldx, heads, d) || !qk_pitch(ldy, heads, d)) return MP_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MP_OK;
    if (!x || !y || !pos || (!wq && q_heads > 0) || (!wk && q_heads < heads) || (x == y && ldx != ldy))
        return MP_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || !aligned16(wq) || !aligned16(wk) || (reinterpret_cast<uintptr_t>(pos) & 3u))
        return MP_ERR_MISALIGNED;
    int sms = 0;
    st = check_device(&sms);
    if (st != MP_OK) return st;
    RopeTable tab{};
    rope_fill(tab, axes, sections, pairs, base, flags);
    QkNormArgs a = qk_args(T, heads, q_heads, d, axes, pairs, eps);
    a.x = reinterpret_cast<const __nv_bfloat16*>(x);
    a.y = reinterpret_cast<__nv_bfloat16*>(y);
    a.wq = reinterpret_cast<const __nv_bfloat16*>(wq);
    a.wk = reinterpret_cast<const __nv_bfloat16*>(wk);
    a.pos = pos;
    a.ldx = ldx;
    a.ldy = ldy;
    const bool wide = qk_wide(d, pairs);
    const int blocks = qk_blocks(a, wide, false);
    const cudaError_t e = qk_dispatch<false>(tab, a, wide, (flags & MP_ROPE_INTERLEAVED) != 0, blocks,
                                             static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

extern "C" size_t mp_qk_norm_rope_bwd_workspace_bytes(int T, int heads, int d) {
    if (T <= 0 || heads <= 0 || d <= 0 || d % 8 != 0 || d > 2 * ROPE_MAX_PAIRS) return 0;
    return static_cast<size_t>(QKN_BWD_ROWS) * 2 * d * sizeof(float);
}

extern "C" mp_status mp_qk_norm_rope_bwd(const mp_bf16* x, const mp_bf16* dy, mp_bf16* dx, const mp_bf16* wq,
                                         const mp_bf16* wk, float* dwq, float* dwk, const int32_t* pos, void* workspace,
                                         size_t workspace_bytes, int T, int heads, int q_heads, int d, long long ldx,
                                         long long lddy, long long lddx, int axes, const int* sections, double base,
                                         float eps, uint32_t flags, void* stream) {
    long long pairs = 0;
    mp_status st = qk_check(T, heads, q_heads, d, axes, sections, base, eps, flags, &pairs);
    if (st != MP_OK) return st;
    if (!qk_pitch(ldx, heads, d) || !qk_pitch(lddy, heads, d) || !qk_pitch(lddx, heads, d))
        return MP_ERR_UNSUPPORTED_SHAPE;
    if ((!dwq && q_heads > 0) || (!dwk && q_heads < heads)) return MP_ERR_INVALID_ARG;
    if (!aligned16(dwq) || !aligned16(dwk)) return MP_ERR_MISALIGNED;
    if (T > 0) {
        if (!x || !dy || !dx || !pos || (!wq && q_heads > 0) || (!wk && q_heads < heads) || (dx == x && lddx != ldx) ||
            (dx == dy && lddx != lddy))
            return MP_ERR_INVALID_ARG;
        if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || !aligned16(wq) || !aligned16(wk) ||
            (reinterpret_cast<uintptr_t>(pos) & 3u))
            return MP_ERR_MISALIGNED;
        if (!workspace || !aligned16(workspace) || workspace_bytes < mp_qk_norm_rope_bwd_workspace_bytes(T, heads, d))
            return MP_ERR_WORKSPACE;
    }
    int sms = 0;
    st = check_device(&sms);
    if (st != MP_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int blocks = 0, q_rows = 0, k_row = 0;
    if (T > 0) {
        RopeTable tab{};
        rope_fill(tab, axes, sections, pairs, base, flags);
        QkNormArgs a = qk_args(T, heads, q_heads, d, axes, pairs, eps);
        a.x = reinterpret_cast<const __nv_bfloat16*>(x);
        a.dy = reinterpret_cast<const __nv_bfloat16*>(dy);
        a.y = reinterpret_cast<__nv_bfloat16*>(dx);
        a.wq = reinterpret_cast<const __nv_bfloat16*>(wq);
        a.wk = reinterpret_cast<const __nv_bfloat16*>(wk);
        a.pos = pos;
        a.sums = static_cast<float*>(workspace);
        a.ldx = ldx;
        a.lddy = lddy;
        a.ldy = lddx;
        const bool wide = qk_wide(d, pairs);
        blocks = qk_blocks(a, wide, true);
        q_rows = a.q_slots > 0 ? a.q_blocks : 0;
        // Keys' rows: those of the blocks that have keys alone, or of all blocks, or none where there is no key head.
        k_row = q_heads == heads || a.k_steps > 0 ? a.q_blocks : 0;
        const cudaError_t e = qk_dispatch<true>(tab, a, wide, (flags & MP_ROPE_INTERLEAVED) != 0, blocks, s);
        if (e != cudaSuccess) return MP_ERR_CUDA;
    }
    // T = 0: no rows, the sums are zero.
    const cudaError_t e = launch_pdl(qk_norm_dw_kernel, dim3(static_cast<unsigned>(2 * ((d + 31) / 32))), dim3(1024), 0, s,
                                     static_cast<const float*>(workspace), dwq, dwk, q_rows, k_row, blocks, d);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
