// Entry point of the rotary positions over several axes: mp_rope_axes.
//
// A head's pair i of elements (a, b) becomes (a cos A - b sin A, b cos A + a sin A) with the
// angle A = pos[axis(i)] * base^-e(i): time, height and width (or any up to four axes) each own a
// run of consecutive pairs. The rotation is orthogonal, so its gradient is the rotation back
// (`inverse`: the angle's sign).
//
// Bound by memory: x is read and y written once. One warp takes one token (or a share of its
// heads when tokens are few): a lane owns VEC neighbouring pairs, computes their sines once and
// walks the heads, so the sines cost about a fifth of the instructions at 32 heads. 28,350 tokens of 40 heads of 96
// (436 MB): 66.5 us, 6.55 TB/s, 97 % of a plain copy's rate; neighbouring pairs, 32 heads of 72: 6.13 TB/s. Five
// tokens: 3 us on the device, less than the call takes on the host.
#include "mptp_internal.h"
#include "mptp_launch.cuh"
#include "mptp_ptx.cuh"
#include "mptp_rope.cuh"

namespace mptp {

constexpr int ROPE_WARPS = 8;        // warps (tokens, or shares of tokens) per block
constexpr int ROPE_UNROLL = 4;       // heads whose loads are in flight together, per lane

struct RopeArgs {
    const __nv_bfloat16* x;
    __nv_bfloat16* y;
    const int32_t* pos;  // [axes][T]
    long long ldx, ldy;
    int T, heads, d;
    int pairs;           // rotated pairs per head
    int shares;          // warps per token
    int sign;            // +1, or -1 for the inverse
};

template <int VEC, bool INTER>
__global__ void __launch_bounds__(ROPE_WARPS * 32) rope_axes_kernel(const __grid_constant__ RopeTable tab,
                                                                    const RopeArgs a) {
    using V = typename RopeVec<VEC>::T;
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * ROPE_WARPS + (threadIdx.x >> 5);
    const int token = static_cast<int>(w / a.shares);
    const int share = static_cast<int>(w % a.shares);
    const int groups = a.pairs / VEC;       // lanes per head (<= 32)
    const int per_warp = 32 / groups;       // heads a warp has in hand at once
    const int g = lane % groups;
    const int sub = lane / groups;
    grid_dependency_wait();
    grid_launch_dependents();
    if (token >= a.T) return;
    const __nv_bfloat16* xr = a.x + token * a.ldx;
    __nv_bfloat16* yr = a.y + token * a.ldy;
    if (sub < per_warp) {
        float c[VEC], s[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int i = g * VEC + j;
            const long long p = static_cast<long long>(a.pos[static_cast<long long>(tab.axis[i]) * a.T + token]) * a.sign;
            rope_sincos(tab, i, p, &s[j], &c[j]);
        }
        const int o0 = INTER ? 2 * VEC * g : VEC * g;
        const int o1 = INTER ? o0 + VEC : o0 + a.pairs;
        const int step = per_warp * a.shares;
        for (int h0 = share * per_warp + sub; h0 < a.heads; h0 += ROPE_UNROLL * step) {
            union {
                V v;
                uint32_t w[VEC / 2];
            } u[ROPE_UNROLL], v[ROPE_UNROLL];
#pragma unroll
            for (int k = 0; k < ROPE_UNROLL; ++k) {
                const int hd = h0 + k * step;
                if (hd < a.heads) {
                    u[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + o0);
                    v[k].v = *reinterpret_cast<const V*>(xr + hd * a.d + o1);
                }
            }
#pragma unroll
            for (int k = 0; k < ROPE_UNROLL; ++k) {
                const int hd = h0 + k * step;
                if (hd < a.heads) {
                    rope_rotate<VEC, INTER>(u[k].w, v[k].w, c, s);
                    *reinterpret_cast<V*>(yr + hd * a.d + o0) = u[k].v;
                    *reinterpret_cast<V*>(yr + hd * a.d + o1) = v[k].v;
                }
            }
        }
    }
    // The part of each head behind the rotated pairs passes through.
    const int rest = a.d - 2 * a.pairs;
    if (rest > 0 && a.x != a.y) {
        const int nv = rest / 4;  // 8-byte pieces
        for (int i = share * 32 + lane; i < a.heads * nv; i += 32 * a.shares) {
            const int o = i / nv * a.d + 2 * a.pairs + i % nv * 4;
            *reinterpret_cast<uint2*>(yr + o) = *reinterpret_cast<const uint2*>(xr + o);
        }
    }
}

template <int VEC, bool INTER>
static cudaError_t launch_rope(const RopeTable& tab, const RopeArgs& a, cudaStream_t s) {
    const long long warps = static_cast<long long>(a.T) * a.shares;
    const long long blocks = (warps + ROPE_WARPS - 1) / ROPE_WARPS;
    const cudaError_t e = launch_pdl(rope_axes_kernel<VEC, INTER>, dim3(static_cast<unsigned>(blocks)),
                                     dim3(ROPE_WARPS * 32), 0, s, tab, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mptp

using namespace mptp;

extern "C" mp_status mp_rope_axes(const mp_bf16* x, mp_bf16* y, const int32_t* pos, int T, int heads, int d,
                                  long long ldx, long long ldy, int axes, const int* sections, double base,
                                  uint32_t flags, void* stream) {
    long long pairs = 0;
    if (T < 0 || heads <= 0 || d <= 0 ||
        !rope_valid(axes, sections, base, flags, MP_ROPE_INTERLEAVED | MP_ROPE_PER_AXIS | MP_ROPE_INVERSE, &pairs))
        return MP_ERR_INVALID_ARG;
    const long long row = static_cast<long long>(heads) * d;
    if (d % 8 != 0 || d > 2 * ROPE_MAX_PAIRS || pairs < 4 || pairs % 4 != 0 || 2 * pairs > d || row > 0x7fffffffLL ||
        ldx < row || ldy < row || ldx % 8 != 0 || ldy % 8 != 0)
        return MP_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MP_OK;
    if (!x || !y || !pos) return MP_ERR_INVALID_ARG;
    if (x == y && ldx != ldy) return MP_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(y) || (reinterpret_cast<uintptr_t>(pos) & 3u)) return MP_ERR_MISALIGNED;
    int sms = 0;
    const mp_status st = check_device(&sms);
    if (st != MP_OK) return st;

    RopeTable tab{};
    rope_fill(tab, axes, sections, pairs, base, flags);
    RopeArgs a{};
    a.x = reinterpret_cast<const __nv_bfloat16*>(x);
    a.y = reinterpret_cast<__nv_bfloat16*>(y);
    a.pos = pos;
    a.ldx = ldx;
    a.ldy = ldy;
    a.T = T;
    a.heads = heads;
    a.d = d;
    a.pairs = static_cast<int>(pairs);
    a.sign = (flags & MP_ROPE_INVERSE) ? -1 : 1;
    // 16-byte pieces where the second half of a head starts on one, else 8-byte pieces.
    const bool wide = pairs % 8 == 0;
    const int heads_in_hand = 32 / static_cast<int>(pairs / (wide ? 8 : 4));
    // A token's heads are shared among warps while that leaves SMs without a warp.
    a.shares = 1;
    while (static_cast<long long>(T) * a.shares < 8LL * sms && a.shares * heads_in_hand < heads) a.shares *= 2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (flags & MP_ROPE_INTERLEAVED)
        e = wide ? launch_rope<8, true>(tab, a, s) : launch_rope<4, true>(tab, a, s);
    else
        e = wide ? launch_rope<8, false>(tab, a, s) : launch_rope<4, false>(tab, a, s);
    return e == cudaSuccess ? MP_OK : MP_ERR_CUDA;
}
