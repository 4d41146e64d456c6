// Entry points of the gated feed-forward block: mp_glu_fwd and mp_glu_bwd.
//
//   [G | U] = X [Wg | Wu],  Y = act(G) * U,  Z = Y Wd        act: SiLU or the erf GeLU
//   dY = dZ Wd^T,  dG = dY * U * act'(G),  dU = dY * act(G)
//   dX = [dG | dU] [Wg | Wu]^T,  dWg = X^T dG,  dWu = X^T dU,  dWd = Y^T dZ
//
// The block is split for tensor parallelism as the GeLU block is ("Megatron-LM: Training
// Multi-Billion Parameter Language Models Using Model Parallelism", section 3.4): shard i owns
// columns [i f/t, (i+1) f/t) of Wg and of Wu and the same rows of Wd. The shards' partial outputs
// (the g sum of Z, the f sum of dX) are added inside the K-loop.
//
// Forward: both projections, the activation and the product are one launch. A CTA pair's tile is
// 256 tokens x (128 gate + 128 up columns of the same outputs): the leader loads gate columns and its
// peer up columns, one tcgen05.mma (M = 256, N = 256) multiplies both, and each epilogue thread finds
// a token's gate and up values in its own TMEM lane, 128 columns apart, in fp32. So G and U are
// rounded only where the caller keeps them for the backward pass; Y comes from the fp32 values.
// Then Z is one row-parallel GEMM over Y. Few tokens take a kernel bound by reading the weights for both
// (mptp_gemm_few.cuh).
// Backward: one GEMM gives dY, whose epilogue reads G and U and writes dG and dU (dY never reaches
// memory); dX, dW and dWd are three GEMMs, side by side where that is shorter (mptp_mlp_host.cuh).
// Roundings to bf16: Y, dG and dU as operands of the next product, which the tensor core wants in 16 bits, and G and U
// between the passes, as U of the GeLU block is: fp32 would add 200 MB to the 500 MB that bound the kernel of dG and dU,
// computing them again in the backward 22 % of a step's products. Each costs what one rounding of the result does: Z and
// dWd are 2.3e-3 of their norm off, dX and dW 3.0e-3, results of fp32 products rounded once 1.7e-3.
// Bound by the tensor core: T = 8192, h = 2304, f = 6144, SiLU, 1.26 to 1.31 ms forward and backward, 1.59 to 1.65 PFLOP/s,
// 93 to 96 % of the library's sustained rate for a plain product. Alone, the launches take 245 us ([G | U] and Y), 120 (Z), 157 (dG
// and dU: 119 without the epilogue, whose gates, ups and gradients are 500 MB beside the K loop), 241, 240 and 122.
#include <algorithm>

#include "mptp_gemm_few.cuh"
#include "mptp_mlp_host.cuh"

using namespace mptp;

namespace {

bool bad_act(int act) { return act != MP_ACT_SILU && act != MP_ACT_GELU; }

// Whether the forward takes the kernel for few tokens. One slice of them always (h = 2304, f = 6144: 20 us for a token,
// 28 for 128, the large tiles 44). More while every slice's blocks of columns have an SM each and the weights stay
// below twice L2's size, so that a slice finds them there: 384 tokens 38 us against 55; h = 1536, f = 4096, 512 tokens
// 28 against 38; h = 1024, f = 2048, 1024 tokens 21 against 30; h = 4096, f = 8192, 256 tokens 55 against 62. Beyond:
// a second round of CTAs takes 62 us against 56 (513 tokens, h = 2304), 400 MB of weights 97 against 87 (256 tokens).
bool few_tokens(int T, int h, int f, int sms) {
    const int slices = ceil_div(T, FEW_SLICE);
    return slices == 1 || (ceil_div(std::max(h, f), 128) <= sms / slices && 6LL * h * f <= (1LL << 28));
}

// The backward takes it up to three slices: h = 2304, f = 6144 50 us against 86 with the large tiles for a token, 63 for
// 128, 88 against 90 for 384, more than 100 against 88 for 512; h = 704, f = 3136 25 against 52, 31, 40 against 55.
constexpr int FEW_BWD_SLICES = 3;

}  // namespace

extern "C" mp_status mp_glu_fwd(const mp_bf16* X, const mp_bf16* W, const mp_bf16* Wd, mp_bf16* Z, mp_bf16* Y,
                                mp_bf16* GU_save, int T, int h, int f, int t, int act, uint32_t* d_status,
                                void* stream) {
    mp_status st = check_mlp_shape(T, h, f, t);
    if (st != MP_OK) return st;
    if (bad_act(act)) return MP_ERR_INVALID_ARG;
    if (f > 0x3fffffff) return MP_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MP_OK;
    if (!X || !W || !Wd || !Z || !Y) return MP_ERR_INVALID_ARG;
    const void* ptrs[] = {X, W, Wd, Z, Y, GU_save};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return MP_ERR_MISALIGNED;
    if (d_status && (reinterpret_cast<uintptr_t>(d_status) & 3u)) return MP_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_device(&sms)) != MP_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const double Tb = 2.0 * T, hb = 2.0 * h;
    const size_t f2 = size_t(2) * f;
    if (few_tokens(T, h, f, sms)) {
        st = launch_gemm_few<FEW_GATED>(X, W, Y, GU_save, T, h, f, static_cast<int>(f2), act, d_status, sms, s);
        return st != MP_OK ? st : launch_gemm_few<FEW_PLAIN>(Y, Wd, Z, nullptr, T, f, h, h, act, d_status, sms, s);
    }

    // [G | U] = X W and Y = act(G) * U, tiles of 128 outputs.
    TmapSet m1{};
    int b1 = 0;
    if (!make_tmap_bf16(&m1.a, X, h, T, h, 64, BM) || !(b1 = make_tmap_mn_operand(&m1.b, W, f2, h, f2)) ||
        !make_tmap_bf16_out(&m1.o0, Y, f, T, f) ||
        (GU_save && (!make_tmap_bf16_out(&m1.o1, GU_save, f, T, f2) || !make_tmap_bf16_out(&m1.o2, GU_save + f, f, T, f2))))
        return MP_ERR_CUDA;
    GemmArgs a1 = launch_args(d_status);
    a1.pr = problem(T, f, 128, 0, h / BK, false, true, Tb * h, 2 * hb * f);
    a1.pr.b_mn = b1;
    a1.has_out1 = GU_save ? 1 : 0;
    a1.act = act;
    a1.glu_f = f;
    if (launch_gelu_epi<EPI_GLU>(m1, a1, sms, s) != cudaSuccess) return MP_ERR_CUDA;

    // Z = sum_i Y_i Wd_i, shards in ascending order in the K-loop (the g sum).
    TmapSet m2{};
    int b2 = 0;
    if (!make_tmap_bf16(&m2.a, Y, f, T, f, 64, BM) || !(b2 = make_tmap_mn_operand(&m2.b, Wd, h, f, h)) ||
        !make_tmap_bf16_out(&m2.o0, Z, h, T, h))
        return MP_ERR_CUDA;
    GemmArgs a2 = launch_args(d_status);
    a2.pr = problem(T, h, 256, 0, f / BK, false, true, Tb * f, hb * f);
    a2.pr.b_mn = b2;
    const bool split2 = use_split<256>(T, h, f / BK, sms);
    if ((split2 ? launch_gemm_split<256, SPLIT_PAIRS>(m2, a2, sms, s) : launch_gemm_tc<256, EPI_STORE, 4>(m2, a2, sms, s)) !=
        cudaSuccess)
        return MP_ERR_CUDA;
    return MP_OK;
}

extern "C" mp_status mp_glu_bwd(const mp_bf16* X, const mp_bf16* W, const mp_bf16* Wd, const mp_bf16* GU,
                                const mp_bf16* Y, const mp_bf16* dZ, mp_bf16* dX, mp_bf16* dW, mp_bf16* dWd,
                                mp_bf16* dGU_ws, int T, int h, int f, int t, int act, uint32_t* d_status,
                                void* stream) {
    mp_status st = check_mlp_shape(T, h, f, t);
    if (st != MP_OK) return st;
    if (bad_act(act)) return MP_ERR_INVALID_ARG;
    if (f > 0x3fffffff) return MP_ERR_UNSUPPORTED_SHAPE;
    if (!W || !Wd || !dW || !dWd) return MP_ERR_INVALID_ARG;
    if (T > 0 && (!X || !GU || !Y || !dZ || !dX || !dGU_ws)) return MP_ERR_INVALID_ARG;
    const void* ptrs[] = {X, W, Wd, GU, Y, dZ, dX, dW, dWd, dGU_ws};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return MP_ERR_MISALIGNED;
    if (d_status && (reinterpret_cast<uintptr_t>(d_status) & 3u)) return MP_ERR_MISALIGNED;
    int sms = 0;
    if ((st = check_device(&sms)) != MP_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t f2 = size_t(2) * f;
    if (T == 0) {
        // Empty batch: the weight gradients are sums over zero tokens.
        if (cudaMemsetAsync(dW, 0, size_t(h) * f2 * 2, s) != cudaSuccess ||
            cudaMemsetAsync(dWd, 0, size_t(f) * h * 2, s) != cudaSuccess)
            return MP_ERR_CUDA;
        return MP_OK;
    }
    const double Tb = 2.0 * T, hb = 2.0 * h;

    // dW = X^T dGU (both operands MN-major).
    TmapSet m5{};
    int a5f = 0, b5f = 0;
    if (!(a5f = make_tmap_mn_operand(&m5.a, X, h, T, h)) || !(b5f = make_tmap_mn_operand(&m5.b, dGU_ws, f2, T, f2)) ||
        !make_tmap_bf16_out(&m5.o0, dW, f2, h, f2))
        return MP_ERR_CUDA;
    GemmArgs a5 = launch_args(d_status);
    a5.pr = problem(h, 2 * f, 256, 0, ceil_div(T, BK), true, true, Tb * h, 2 * Tb * f);
    a5.pr.a_mn = a5f;
    a5.pr.b_mn = b5f;

    // dWd = Y^T dZ (both operands MN-major).
    TmapSet m6{};
    int a6f = 0, b6f = 0;
    if (!(a6f = make_tmap_mn_operand(&m6.a, Y, f, T, f)) || !(b6f = make_tmap_mn_operand(&m6.b, dZ, h, T, h)) ||
        !make_tmap_bf16_out(&m6.o0, dWd, h, f, h))
        return MP_ERR_CUDA;
    GemmArgs a6 = launch_args(d_status);
    a6.pr = problem(f, h, 256, 0, ceil_div(T, BK), true, true, Tb * f, Tb * h);
    a6.pr.a_mn = a6f;
    a6.pr.b_mn = b6f;
    if (T <= FEW_BWD_SLICES * FEW_SLICE && few_tokens(T, h, f, sms)) {
        // dY with dG, dU, then dX by the kernel for few tokens. The weights' gradients are bound by their stores: eight
        // epilogue warps, h = 2304, f = 6144, one token 50.5 us for all four launches against 57.7 with four.
        st = launch_gemm_few<FEW_DGLU>(dZ, Wd, dGU_ws, const_cast<mp_bf16*>(GU), T, h, f, h, act, d_status, sms, s);
        if (st == MP_OK)
            st = launch_gemm_few<FEW_PLAIN_T>(dGU_ws, W, dX, nullptr, T, static_cast<int>(f2), h, static_cast<int>(f2), act,
                                              d_status, sms, s);
        if (st != MP_OK) return st;
        return launch_gemm_tc<256, EPI_STORE, 8>(m5, a5, sms, s) == cudaSuccess &&
                       launch_gemm_tc<256, EPI_STORE, 8>(m6, a6, sms, s) == cudaSuccess
                   ? MP_OK
                   : MP_ERR_CUDA;
    }

    // dY = dZ Wd^T; dG, dU in its epilogue.
    TmapSet m3{};
    if (!make_tmap_bf16(&m3.a, dZ, h, T, h, 64, BM) || !make_tmap_bf16(&m3.b, Wd, h, f, h, 64, 128) ||
        !make_tmap_bf16_out(&m3.o0, dGU_ws, f, T, f2) || !make_tmap_bf16_out(&m3.o1, dGU_ws + f, f, T, f2) ||
        !make_tmap_bf16_out(&m3.x0, GU, f, T, f2) || !make_tmap_bf16_out(&m3.x1, GU + f, f, T, f2))
        return MP_ERR_CUDA;
    GemmArgs a3 = launch_args(d_status);
    a3.pr = problem(T, f, 256, 0, h / BK, false, false, Tb * h, 2.0 * f * h);
    a3.act = act;
    if (launch_gemm_tc<256, EPI_DGLU, 4>(m3, a3, sms, s) != cudaSuccess) return MP_ERR_CUDA;

    // dX = dGU W^T: gate blocks, then up blocks, shards ascending in each (the f sum). Tiles of 224 or 256
    // columns, whichever makes the rounds of CTA pairs times the width less (h = 2304, T = 8192: 4 rounds of
    // 256 against 5 of 224, the training step 1287 against 1305 us). Narrower tiles do not help where few rows
    // leave pairs idle: 128-wide ones took the same time a K block, the producer's two loads.
    const int pairs = resident_pairs<256, EPI_STORE, 4>(sms);
    auto k4_cost = [&](int bn) { return (tiles_of(T, h, bn) + pairs - 1) / pairs * bn; };
    const int bn4 = k4_cost(K4_BN) < k4_cost(256) ? K4_BN : 256;
    TmapSet m4{};
    if (!make_tmap_bf16(&m4.a, dGU_ws, f2, T, f2, 64, BM) || !make_tmap_bf16(&m4.b, W, f2, h, f2, 64, bn4 / 2) ||
        !make_tmap_bf16_out(&m4.o0, dX, h, T, h))
        return MP_ERR_CUDA;
    GemmArgs a4 = launch_args(d_status);
    a4.pr = problem(T, h, bn4, 0, 2 * (f / BK), false, false, 2 * Tb * f, 2 * hb * f);

    return launch_grad_gemms(m4, a4, bn4, W, static_cast<int>(f2), m5, a5, m6, a6, sms, s);
}
