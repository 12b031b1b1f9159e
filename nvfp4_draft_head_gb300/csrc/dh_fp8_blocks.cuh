// Quantisation of activations to FP8 (E4M3) with one scale per token and 128 features, and what
// the two product kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dh_gemm.cuh"
#include "dh_rows.cuh"

namespace dh {
namespace f8 {

constexpr int kBlock = 128;   // elements of a scale

// The scale of a block from the bits of its largest magnitude (NaN and infinities on top): NaN
// for a block with a value that is not finite.
__device__ __forceinline__ float block_scale(uint32_t top) {
    return top < 0x7F800000u ? act_fp8_scale(__uint_as_float(top)) : __uint_as_float(0x7FC00000u);
}

// 16 elements of a block held by eight lanes (n of them there): their codes, and the block's
// scale, the same in all eight lanes.
template <class T, bool VEC>
__device__ __forceinline__ float encode16(const T* src, int n, uint4& codes) {
    float v[16];
    if (n == 16) {
        rows::load16<T, VEC>(src, v);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? rows::Elem<T>::load(src + i) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float s = block_scale(top);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = fminf(fmaxf(__fdiv_rn(v[4 * i + j], s), -448.0f), 448.0f);
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    codes = make_uint4(w[0], w[1], w[2], w[3]);
    return s;
}

inline bool rows_aligned16(const void* x, long long ld_bytes, int rows) {
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (rows == 1 || ld_bytes % 16 == 0);
}

// Products of up to kFewTokens tokens (dh_fp8_few.cu); scales null: x is quantised in the kernel.
constexpr int kFewTokens = 128, kFusedTokens = 16;
// Whether that form can take a product (its share of the steps fits a CTA), and about how long
// it would be.
bool few_supported(const Fp8BlockArgs& f, float* us);
// Whether its fused form can take a product of this many steps, by the sizes alone: such a product
// needs no workspace.
bool fused_fits(int steps);
cudaError_t launch_few(const Fp8BlockArgs& f, const uint8_t* codes, int ldc, const float* scales, cudaStream_t s);

}  // namespace f8
}  // namespace dh
