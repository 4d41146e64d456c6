// What the write, the read and the attention over the 8-bit cache share: the pool of pages and its checks.
//
// A page holds `page` tokens of one sequence for every key head, head by head: [kv_heads][page][d] e4m3 codes, so a
// head's tokens are one contiguous run, and one scale a head. A value is code * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mptp_internal.h"
#include "mptp_ptx.cuh"

namespace mptp {

constexpr uint32_t KV_SEQ_RANGE = MP_DEV_SEQ_RANGE;
constexpr uint32_t KV_PAGE_RANGE = MP_DEV_PAGE_RANGE;

struct KvPool {
    uint8_t* codes[2];  // keys, values
    float* scales[2];
    long long ld_codes[2], ld_scales[2];  // from page to page
    uint32_t pitch16[2], pitch_scales[2];  // the same in 16-byte pieces and in floats
    const int32_t* table;                 // [nseq][max_pages]
    int pages, max_pages, page, kv_heads, d;
    int page_shift;                       // log2 of the page
    __device__ __forceinline__ uint8_t* head_codes(int kind, long long id, int head) const {
        return (kind ? codes[1] + id * ld_codes[1] : codes[0] + id * ld_codes[0]) + static_cast<long long>(head) * page * d;
    }
    __device__ __forceinline__ float* head_scale(int kind, long long id, int head) const {
        return (kind ? scales[1] + id * ld_scales[1] : scales[0] + id * ld_scales[0]) + head;
    }
};

// The lower two codes as two halves (exact: every e4m3 value is a half).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(two));
    return r;
}
// The same of the upper two of four.
__device__ __forceinline__ uint32_t e4m3x2_hi_to_f16x2(uint32_t four) {
    uint32_t r;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(four));
    return r;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two floats as e4m3 codes, `lo` in the low byte; beyond 448 they stay at 448, NaN stays NaN.
__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{.reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %2, %1; cvt.u32.u16 %0, t;}" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

// The pool's pointers, after kv_pool_sizes.
inline mp_status kv_pool_pointers(const void* kc, const void* vc, const void* ks, const void* vs, const void* table) {
    if (!kc || !vc || !ks || !vs || !table) return MP_ERR_INVALID_ARG;
    auto word = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; };
    return aligned16(kc) && aligned16(vc) && word(ks) && word(vs) && word(table) ? MP_OK : MP_ERR_MISALIGNED;
}

// The pool's sizes that every entry point takes.
inline bool kv_pool_sizes(int pages, int max_pages, int page, int kv_heads, int d, long long ld_kc, long long ld_vc,
                          long long ld_ks, long long ld_vs) {
    const long long row = static_cast<long long>(kv_heads) * page * d;
    return (page == 16 || page == 32 || page == 64 || page == 128) && pages >= 1 && max_pages >= 1 &&
           static_cast<long long>(max_pages) * page <= 0x7fffff00LL && static_cast<long long>(kv_heads) * d <= 0x7fffffffLL &&
           ld_kc >= row && ld_vc >= row && ld_kc % 16 == 0 && ld_vc % 16 == 0 && ld_ks >= kv_heads && ld_vs >= kv_heads &&
           (ld_kc | ld_vc) >> 36 == 0 && (ld_ks | ld_vs) >> 32 == 0;
}

}  // namespace mptp
