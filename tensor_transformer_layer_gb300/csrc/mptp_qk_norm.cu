// Entry points of the norm of queries and keys with their rotation: mp_qk_norm_rope, mp_qk_norm_rope_bwd.
//
// Per head of d elements, with r = 1 / sqrt(mean(x^2) + eps) and n = x r:
//   forward   y = R(w * n), R the rotation of mp_rope_axes (w: the queries' or the keys' weight)
//   backward  g = R^-1 dy,  dw = sum over tokens and heads of g * n,
//             dx = r (w * g - n mean(w * g * n))
// r is computed again from x, which the backward pass reads anyway: nothing is kept between the two.
//
// Bound by memory: x once in and y once out; backward x and dy in and dx out. A warp takes a token (or a share of its
// heads where tokens are few): a head lies across G = d / (2 VEC) lanes, VEC rotated pairs in each, or as many
// unrotated elements (cosine 1, sine 0), so that the sums of squares are a few shuffles within the G lanes and the
// angles' sines are computed once for all heads of the token. All of it is fp32 in registers; each output is rounded once.
// The weights' gradients: a lane keeps its columns' sums in registers over all its tokens, a block adds its lanes' in
// shared memory and writes one row of the workspace, a second kernel adds the rows: fixed order, no atomics.
#include "mptp_internal.h"
#include "mptp_launch.cuh"
#include "mptp_ptx.cuh"
#include "mptp_rope.cuh"

namespace mptp {

constexpr int QKN_WARPS = 8;
constexpr int QKN_UNROLL = 4;        // forward: heads in flight per lane
constexpr int QKN_BWD_UNROLL = 2;    // backward: two vectors more of each
constexpr int QKN_BWD_BLOCKS = 304;  // two blocks on each of 152 SMs: the rows of the workspace

struct QkNormArgs {
    const __nv_bfloat16* x;
    const __nv_bfloat16* dy;
    __nv_bfloat16* y;  // backward: dx
    const __nv_bfloat16* wq;
    const __nv_bfloat16* wk;
    const int32_t* pos;  // [axes][T]
    float* sums;         // [blocks][2][d]
    long long ldx, ldy, lddy;
    int T, heads, q_heads, d, pairs, shares;
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

// Sum over the `groups` lanes of a head, in all of them; every lane of the warp takes part.
template <int N>
__device__ __forceinline__ void qk_head_sum(float (&v)[N], int groups, int g, int lane) {
    if ((groups & (groups - 1)) == 0) {
        for (int off = groups >> 1; off > 0; off >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
        return;
    }
    for (int off = 1; off < groups; off <<= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float o = __shfl_down_sync(0xffffffffu, v[k], off);
            if (g + off < groups) v[k] += o;
        }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], lane - g);
}

template <int VEC>
__device__ __forceinline__ void qk_unpack(const uint32_t (&u)[VEC / 2], const uint32_t (&v)[VEC / 2],
                                          float (&f)[2 * VEC]) {
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
        f[2 * j] = rope_lo(u[j]);
        f[2 * j + 1] = rope_hi(u[j]);
        f[VEC + 2 * j] = rope_lo(v[j]);
        f[VEC + 2 * j + 1] = rope_hi(v[j]);
    }
}

// The pairs of a lane turned by the angles of (c, s).
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_turn(float (&f)[2 * VEC], const float (&c)[VEC], const float (&s)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : j + VEC;
        const float a = f[ia], b = f[ib];
        f[ia] = a * c[j] - b * s[j];
        f[ib] = b * c[j] + a * s[j];
    }
}

template <int VEC>
union QkVec {
    typename RopeVec<VEC>::T v;
    uint32_t w[VEC / 2];
};

template <int VEC, bool INTER>
__device__ __forceinline__ void qk_angles(const RopeTable& tab, const QkNormArgs& a, const QkLane<VEC, INTER>& L,
                                          int token, int sign, float (&c)[VEC], float (&s)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        c[j] = 1.0f;
        s[j] = 0.0f;
    }
    if (!L.turns) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const int i = L.g * VEC + j;
        const long long p = a.pos[static_cast<long long>(tab.axis[i]) * a.T + token];
        rope_sincos(tab, i, p * sign, &s[j], &c[j]);
    }
}

// A lane's elements of a weight, packed; zeros where the call has none of its heads.
template <int VEC, bool INTER>
__device__ __forceinline__ void qk_weight(const __nv_bfloat16* w, const QkLane<VEC, INTER>& L, QkVec<VEC>& u, QkVec<VEC>& v) {
    using V = typename RopeVec<VEC>::T;
    u.v = V{};
    v.v = V{};
    if (w != nullptr) {
        u.v = *reinterpret_cast<const V*>(w + L.o0);
        v.v = *reinterpret_cast<const V*>(w + L.o1);
    }
}

template <int VEC, bool INTER>
__global__ void __launch_bounds__(QKN_WARPS * 32) qk_norm_kernel(const __grid_constant__ RopeTable tab,
                                                                 const QkNormArgs a) {
    using V = typename RopeVec<VEC>::T;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * QKN_WARPS + (threadIdx.x >> 5);
    const int token = static_cast<int>(w / a.shares);
    const int share = static_cast<int>(w % a.shares);
    const QkLane<VEC, INTER> L(a.d, a.pairs, lane);
    grid_dependency_wait();
    grid_launch_dependents();
    if (token >= a.T) return;
    const __nv_bfloat16* xr = a.x + token * a.ldx;
    __nv_bfloat16* yr = a.y + token * a.ldy;
    QkVec<VEC> wq[2], wk[2];
    qk_weight(a.wq, L, wq[0], wq[1]);
    qk_weight(a.wk, L, wk[0], wk[1]);
    float c[VEC], s[VEC];
    qk_angles(tab, a, L, token, 1, c, s);
    const int step = L.per_warp * a.shares;
    for (int base = share * L.per_warp; base < a.heads; base += QKN_UNROLL * step) {
        QkVec<VEC> u[QKN_UNROLL], v[QKN_UNROLL];
        float ss[QKN_UNROLL];
#pragma unroll
        for (int k = 0; k < QKN_UNROLL; ++k) {
            const int hd = base + L.sub + k * step;
            u[k].v = V{};
            v[k].v = V{};
            if (L.live && hd < a.heads) {
                u[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + L.o0);
                v[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + L.o1);
            }
        }
#pragma unroll
        for (int k = 0; k < QKN_UNROLL; ++k) {
            float f[2 * VEC];
            qk_unpack<VEC>(u[k].w, v[k].w, f);
            ss[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2 * VEC; ++j) ss[k] += f[j] * f[j];
        }
        qk_head_sum(ss, L.groups, L.g, lane);
#pragma unroll
        for (int k = 0; k < QKN_UNROLL; ++k) {
            const int hd = base + L.sub + k * step;
            const bool q = hd < a.q_heads;
            const float r = rsqrtf(ss[k] * a.inv_d + a.eps);
            float f[2 * VEC], wf[2 * VEC];
            QkVec<VEC> w0, w1;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                w0.w[j] = q ? wq[0].w[j] : wk[0].w[j];
                w1.w[j] = q ? wq[1].w[j] : wk[1].w[j];
            }
            qk_unpack<VEC>(u[k].w, v[k].w, f);
            qk_unpack<VEC>(w0.w, w1.w, wf);
#pragma unroll
            for (int j = 0; j < 2 * VEC; ++j) f[j] = f[j] * r * wf[j];
            qk_turn<VEC, INTER>(f, c, s);
            if (L.live && hd < a.heads) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    u[k].w[j] = rope_pack(f[2 * j], f[2 * j + 1]);
                    v[k].w[j] = rope_pack(f[VEC + 2 * j], f[VEC + 2 * j + 1]);
                }
                *reinterpret_cast<V*>(yr + hd * a.d + L.o0) = u[k].v;
                *reinterpret_cast<V*>(yr + hd * a.d + L.o1) = v[k].v;
            }
        }
    }
}

template <int VEC, bool INTER>
__global__ void __launch_bounds__(QKN_WARPS * 32, 2) qk_norm_bwd_kernel(const __grid_constant__ RopeTable tab,
                                                                        const QkNormArgs a) {
    using V = typename RopeVec<VEC>::T;
    constexpr int U = QKN_BWD_UNROLL;
    // [warp, sub][queries', keys'][d]: 32 lanes of 2 VEC columns a warp and kind
    __shared__ float red[QKN_WARPS * 32 * 2 * VEC * 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const QkLane<VEC, INTER> L(a.d, a.pairs, lane);
    grid_dependency_wait();
    grid_launch_dependents();
    QkVec<VEC> wq[2], wk[2];
    qk_weight(a.wq, L, wq[0], wq[1]);
    qk_weight(a.wk, L, wk[0], wk[1]);
    float aq[2 * VEC], ak[2 * VEC];
#pragma unroll
    for (int j = 0; j < 2 * VEC; ++j) aq[j] = ak[j] = 0.0f;
    const long long items = static_cast<long long>(a.T) * a.shares;
    for (long long w = static_cast<long long>(blockIdx.x) * QKN_WARPS + warp; w < items;
         w += static_cast<long long>(gridDim.x) * QKN_WARPS) {
        const int token = static_cast<int>(w / a.shares);
        const int share = static_cast<int>(w % a.shares);
        const __nv_bfloat16* xr = a.x + token * a.ldx;
        const __nv_bfloat16* gr = a.dy + token * a.lddy;
        __nv_bfloat16* dr = a.y + token * a.ldy;
        float c[VEC], s[VEC];
        qk_angles(tab, a, L, token, -1, c, s);
        const int step = L.per_warp * a.shares;
        for (int base = share * L.per_warp; base < a.heads; base += U * step) {
            QkVec<VEC> x0[U], x1[U], g0[U], g1[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hd = base + L.sub + k * step;
                x0[k].v = x1[k].v = g0[k].v = g1[k].v = V{};
                if (L.live && hd < a.heads) {
                    x0[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + L.o0);
                    x1[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + L.o1);
                    g0[k].v = *reinterpret_cast<const V*>(gr + hd * a.d + L.o0);
                    g1[k].v = *reinterpret_cast<const V*>(gr + hd * a.d + L.o1);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hd = base + L.sub + k * step;
                const bool q = hd < a.q_heads;
                float x[2 * VEC], g[2 * VEC], wf[2 * VEC];
                QkVec<VEC> w0, w1;
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    w0.w[j] = q ? wq[0].w[j] : wk[0].w[j];
                    w1.w[j] = q ? wq[1].w[j] : wk[1].w[j];
                }
                qk_unpack<VEC>(x0[k].w, x1[k].w, x);
                qk_unpack<VEC>(g0[k].w, g1[k].w, g);
                qk_unpack<VEC>(w0.w, w1.w, wf);
                qk_turn<VEC, INTER>(g, c, s);
                float sum[2] = {0.0f, 0.0f};  // x^2, w g x
#pragma unroll
                for (int j = 0; j < 2 * VEC; ++j) {
                    sum[0] += x[j] * x[j];
                    wf[j] *= g[j];
                    sum[1] += wf[j] * x[j];
                }
                qk_head_sum(sum, L.groups, L.g, lane);
                const float r = rsqrtf(sum[0] * a.inv_d + a.eps);
                const float m = sum[1] * a.inv_d * r;  // mean(w g n)
#pragma unroll
                for (int j = 0; j < 2 * VEC; ++j) {
                    const float n = x[j] * r;
                    const float gn = g[j] * n;
                    if (q)
                        aq[j] += gn;
                    else
                        ak[j] += gn;
                    wf[j] = r * (wf[j] - n * m);
                }
                if (L.live && hd < a.heads) {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) {
                        x0[k].w[j] = rope_pack(wf[2 * j], wf[2 * j + 1]);
                        x1[k].w[j] = rope_pack(wf[VEC + 2 * j], wf[VEC + 2 * j + 1]);
                    }
                    *reinterpret_cast<V*>(dr + hd * a.d + L.o0) = x0[k].v;
                    *reinterpret_cast<V*>(dr + hd * a.d + L.o1) = x1[k].v;
                }
            }
        }
    }
    if (L.live) {
        float* row = red + (warp * L.per_warp + L.sub) * 2 * a.d;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            row[L.o0 + j] = aq[j];
            row[L.o1 + j] = aq[VEC + j];
            row[a.d + L.o0 + j] = ak[j];
            row[a.d + L.o1 + j] = ak[VEC + j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += QKN_WARPS * 32) {
        float t = 0.0f;
        for (int k = 0; k < QKN_WARPS * L.per_warp; ++k) t += red[k * 2 * a.d + i];
        a.sums[static_cast<long long>(blockIdx.x) * 2 * a.d + i] = t;
    }
}

// dwq and dwk from the blocks' rows: a block takes 32 of the 2 d columns, eight warps a share of the rows each.
__global__ void __launch_bounds__(256) qk_norm_dw_kernel(const float* sums, float* dwq, float* dwk, int rows, int d) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    grid_launch_dependents();
    float t = 0.0f;
    if (col < 2 * d)
        for (int r = warp; r < rows; r += 8) t += sums[static_cast<long long>(r) * 2 * d + col];
    red[warp][lane] = t;
    __syncthreads();
    if (warp != 0 || col >= 2 * d) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) t += red[k][lane];
    float* out = col < d ? dwq : dwk;
    if (out != nullptr) out[col < d ? col : col - d] = t;
}

// The lanes' vectors are 16 bytes where each half of a head and what is not rotated divide into them, else 8.
static bool qk_wide(int d, long long pairs) { return d % 16 == 0 && pairs % 8 == 0; }

// Warps that share a token's heads: doubled while there would be fewer than eight warps on each of 152 SMs.
static int qk_shares(int T, int heads, int d, bool wide) {
    const int in_hand = 32 / (d / (wide ? 16 : 8));
    int shares = 1;
    while (static_cast<long long>(T) * shares < 8LL * 152 && shares * in_hand < heads) shares *= 2;
    return shares;
}

static int qk_bwd_blocks(int T, int shares) {
    const long long blocks = (static_cast<long long>(T) * shares + QKN_WARPS - 1) / QKN_WARPS;
    return static_cast<int>(blocks < QKN_BWD_BLOCKS ? blocks : QKN_BWD_BLOCKS);
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

static QkNormArgs qk_args(int T, int heads, int q_heads, int d, long long pairs, float eps) {
    QkNormArgs a{};
    a.T = T;
    a.heads = heads;
    a.q_heads = q_heads;
    a.d = d;
    a.pairs = static_cast<int>(pairs);
    a.shares = qk_shares(T, heads, d, qk_wide(d, pairs));
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
    QkNormArgs a = qk_args(T, heads, q_heads, d, pairs, eps);
    a.x = reinterpret_cast<const __nv_bfloat16*>(x);
    a.y = reinterpret_cast<__nv_bfloat16*>(y);
    a.wq = reinterpret_cast<const __nv_bfloat16*>(wq);
    a.wk = reinterpret_cast<const __nv_bfloat16*>(wk);
    a.pos = pos;
    a.ldx = ldx;
    a.ldy = ldy;
    const bool inter = (flags & MP_ROPE_INTERLEAVED) != 0;
    auto kernel = qk_wide(d, pairs) ? (inter ? qk_norm_kernel<8, true> : qk_norm_kernel<8, false>)
                                    : (inter ? qk_norm_kernel<4, true> : qk_norm_kernel<4, false>);
    const long long blocks = (static_cast<long long>(T) * a.shares + QKN_WARPS - 1) / QKN_WARPS;
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(QKN_WARPS * 32), 0,
                                     static_cast<cudaStream_t>(stream), tab, a);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}

extern "C" size_t mp_qk_norm_rope_bwd_workspace_bytes(int T, int heads, int d) {
    if (T <= 0 || heads <= 0 || d <= 0 || d % 8 != 0 || d > 2 * ROPE_MAX_PAIRS) return 0;
    // narrow vectors hold fewer heads, so they never take fewer shares than wide ones
    return static_cast<size_t>(qk_bwd_blocks(T, qk_shares(T, heads, d, false))) * 2 * d * sizeof(float);
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
    int blocks = 0;
    if (T > 0) {
        RopeTable tab{};
        rope_fill(tab, axes, sections, pairs, base, flags);
        QkNormArgs a = qk_args(T, heads, q_heads, d, pairs, eps);
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
        blocks = qk_bwd_blocks(T, a.shares);
        const bool inter = (flags & MP_ROPE_INTERLEAVED) != 0;
        auto kernel = qk_wide(d, pairs) ? (inter ? qk_norm_bwd_kernel<8, true> : qk_norm_bwd_kernel<8, false>)
                                        : (inter ? qk_norm_bwd_kernel<4, true> : qk_norm_bwd_kernel<4, false>);
        const cudaError_t e =
            launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(QKN_WARPS * 32), 0, s, tab, a);
        if (e != cudaSuccess) return MP_ERR_CUDA;
    }
    // T = 0: no rows, the sums are zero.
    const cudaError_t e = launch_pdl(qk_norm_dw_kernel, dim3(static_cast<unsigned>((2 * d + 31) / 32)), dim3(256), 0, s,
                                     static_cast<const float*>(workspace), dwq, dwk, blocks, d);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
