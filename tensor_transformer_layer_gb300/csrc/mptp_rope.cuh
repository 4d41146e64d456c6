// What the rotation and the norm with the rotation share: the frequencies' table and a lane's vectors of pairs.
//
// Angles. A far position times a frequency loses its fraction of a turn in 32-bit floats
// (position 4e6 at one radian a step: half a radian of rounding), and 64-bit float arithmetic is
// slow here. So the frequency is kept in turns as a 64-bit binary fraction F = base^-e / (2 pi),
// and pos * F modulo 2^64 is the exact fraction of a turn that the position stands for: one
// 64-bit integer product, whose top 32 bits go to sincospif. F is within 2^-53 of the frequency
// (the host's double), so at position 2^31 the angle is off by less than 2^-21 turns, and the
// conversion to float adds 2^-25 turns. (For a base below 1, 1 / base times that.)
#pragma once

#include <cuda_bf16.h>

#include <cmath>

#include "mptp.h"

namespace mptp {

constexpr int ROPE_MAX_PAIRS = 128;  // d <= 256
constexpr int ROPE_MAX_AXES = 4;

struct RopeTable {
    unsigned long long turns[ROPE_MAX_PAIRS];  // fraction of a turn per position step, times 2^64
    unsigned char axis[ROPE_MAX_PAIRS];
};

// The flags, axes, sections and base that the entry points share: false where one of them is refused. `pairs`: the
// sections' sum.
inline bool rope_valid(int axes, const int* sections, double base, uint32_t flags, uint32_t allowed, long long* pairs) {
    if (axes < 1 || axes > ROPE_MAX_AXES || !sections || !(base > 0.0) || !std::isfinite(base) || (flags & ~allowed))
        return false;
    *pairs = 0;
    for (int i = 0; i < axes; ++i) {
        if (sections[i] < 0) return false;
        *pairs += sections[i];
    }
    return true;
}

inline void rope_fill(RopeTable& tab, int axes, const int* sections, long long pairs, double base, uint32_t flags) {
    int i = 0;
    for (int ax = 0; ax < axes; ++ax)
        for (int j = 0; j < sections[ax]; ++j, ++i) {
            const double e = (flags & MP_ROPE_PER_AXIS) ? static_cast<double>(j) / sections[ax]
                                                        : static_cast<double>(i) / static_cast<double>(pairs);
            // base < 1 turns faster than one radian a step: only the fraction of a turn matters, of which the double
            // has lost what the frequency's whole turns take (at position 2^31: 1.4e-7 turns at base 0.5, 7.9e-6 at
            // 0.01, 1.2e-3 at 1e-4; 7e-8 at most from base 1 on).
            double f = std::pow(base, -e) * 0.15915494309189533577;
            f -= std::floor(f);
            const double scaled = std::ldexp(f, 64);
            tab.turns[i] = scaled >= 18446744073709551615.0 ? 0ull : static_cast<unsigned long long>(scaled);
            tab.axis[i] = static_cast<unsigned char>(ax);
        }
}

// Sine and cosine of the angle of pair i at position `p`.
__device__ __forceinline__ void rope_sincos(const RopeTable& tab, int i, long long p, float* s, float* c) {
    const unsigned long long turn = static_cast<unsigned long long>(p) * tab.turns[i];
    // top 32 bits as a signed fraction of a turn in [-1/2, 1/2); sincospif takes half turns
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, s, c);
}

// VEC pairs of a lane as fp32, from the two halves of a head or from neighbouring elements.
template <int VEC>
struct RopeVec;
template <>
struct RopeVec<8> {
    using T = uint4;
};
template <>
struct RopeVec<4> {
    using T = uint2;
};

__device__ __forceinline__ float rope_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rope_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t rope_pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// A lane's 2 * VEC elements of one head: two vectors, VEC pairs.
//   half-split:  u holds elements [VEC g, +VEC), v the same of the second half (at + pairs)
//   interleaved: u, v hold elements [2 VEC g, +2 VEC): word j is pair j
template <int VEC, bool INTER>
__device__ __forceinline__ void rope_rotate(uint32_t (&u)[VEC / 2], uint32_t (&v)[VEC / 2], const float (&c)[VEC],
                                            const float (&s)[VEC]) {
    if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            uint32_t& w = j < VEC / 2 ? u[j % (VEC / 2)] : v[j % (VEC / 2)];
            const float a = rope_lo(w), b = rope_hi(w);
            w = rope_pack(a * c[j] - b * s[j], b * c[j] + a * s[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            const float a0 = rope_lo(u[j]), a1 = rope_hi(u[j]), b0 = rope_lo(v[j]), b1 = rope_hi(v[j]);
            const float c0 = c[2 * j], c1 = c[2 * j + 1], s0 = s[2 * j], s1 = s[2 * j + 1];
            u[j] = rope_pack(a0 * c0 - b0 * s0, a1 * c1 - b1 * s1);
            v[j] = rope_pack(b0 * c0 + a0 * s0, b1 * c1 + a1 * s1);
        }
    }
}

}  // namespace mptp
