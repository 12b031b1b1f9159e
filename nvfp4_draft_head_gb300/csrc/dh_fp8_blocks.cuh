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

// Rows of activations: [M][width] of T, ld elements apart.
template <class T>
struct Rows {
    const T* x;
    long long ld;
    int M, width;
    __device__ __forceinline__ const T* at(int m, int k) const { return x + static_cast<size_t>(m) * ld + k; }
    __device__ __forceinline__ const T* end() const { return at(M - 1, width); }
};

// 16 elements at p, which lie at any address: the 16-byte vectors that cover them, shifted (one
// load per element made the quantiser of 4,912 x 13,925 three times as long). At the matrix's
// ends, where a vector would reach beyond it, element by element.
template <class T>
__device__ __forceinline__ void load16_any(const T* p, const Rows<T>& rows, float (&v)[16]) {
    constexpr int kVecs = static_cast<int>(sizeof(T)) + 1, kWords = 4 * kVecs;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), first = at & ~static_cast<uintptr_t>(15);
    if (first < reinterpret_cast<uintptr_t>(rows.x) || first + 16 * kVecs > reinterpret_cast<uintptr_t>(rows.end())) {
        dh::rows::load16<T, false>(p, v);
        return;
    }
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(first)[i];
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
    const uint32_t off = static_cast<uint32_t>(at & 15);
#pragma unroll
    for (int b = 1; b <= 2; b <<= 1)   // whole words
#pragma unroll
        for (int i = 0; i + b < kWords; ++i) w[i] = off & (4 * b) ? w[i + b] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
    }
#pragma unroll
    for (int i = 0; i < 16; i += dh::rows::Elem<T>::kVec) {
        constexpr int kPer = 4 * static_cast<int>(sizeof(T));   // words of 16 elements
        const int k = i * kPer / 16;
        dh::rows::Elem<T>::unpack(make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]), reinterpret_cast<float(&)[dh::rows::Elem<T>::kVec]>(v[i]));
    }
}

// v / s, rounded to nearest, from inv = 1 / s so rounded: by Markstein's theorem one correction of
// v inv by its exact remainder. (Compared with the IEEE division for every significand of s at
// E4M3's ties and three neighbours on each side: no difference. Where the remainder underflows, v
// is below 2^-100, and its code 0 either way.) Three operations an element in place of a
// division's dozen: 1 x 4,608 x 2,560, quantised in the product's kernel, 8.5 us with divisions, 6.1;
// the quantiser of 2,048 x 2,560 8.2 and 7.0.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return fmaf(fmaf(-q, s, v), inv, q);
}

// 16 elements of row m from k, of a block held by eight lanes (n of them there): their codes, and
// the block's scale, the same in all eight lanes.
template <class T, bool VEC>
__device__ __forceinline__ float encode16(const Rows<T>& rows, int m, int k, int n, uint4& codes) {
    const T* src = rows.at(m, k);
    float v[16];
    if (n == 16) {
        if constexpr (VEC) dh::rows::load16<T, true>(src, v);
        else load16_any<T>(src, rows, v);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = i < n ? dh::rows::Elem<T>::load(src + i) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const float s = block_scale(top), inv = __frcp_rn(s);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = quotient(v[4 * i + j], s, inv);   // (the conversion clamps)
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

// Products of up to kFewTokens tokens (dh_fp8_few.cuh): tokens that a tile has columns for, the CTAs
// of a cluster that share the contraction (0: not in this form), whether the activations are
// quantised in the kernel, and about how long it takes.
constexpr int kFewTokens = 64;
struct FewPlan {
    int columns, splits;
    bool fused;
    float us;
};
FewPlan few_plan(int M, int out, int width);
template <class TY>
cudaError_t launch_few(const Fp8BlockArgs& f, const FewPlan& plan, const uint8_t* codes, int ldc, const float* scales, cudaStream_t s);

}  // namespace f8
}  // namespace dh
