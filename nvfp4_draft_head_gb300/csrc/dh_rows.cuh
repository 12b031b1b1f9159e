// Helpers of the operators on rows of logits (token log-probabilities,
// distillation): element types, a row's split into 16-byte vectors over the
// CTAs of a cluster, its asynchronous stream through shared memory, and the
// running softmax statistics.
//
// Statistics of a set of logits z, at temperature t with c = log2(e) / t, all in
// 32 bits: m = max z, s = sum 2^(z c - mc), s1 = sum 2^(z c - mc) (z c - mc),
// where mc is m c rounded. One multiply-add per logit gives the exponent with a
// single rounding; that mc is off m c by r = m c - mc (exact from one
// multiply-add) is a common factor 2^r, taken off at the end: with S the sum
// of e^((z - m) / t), ln S = ln s - r ln 2. Two sets are joined by moving
// both to the larger maximum: s' = 2^D s and s1' = 2^D (s1 + D s), D = mc - mc'.
//
// That form needs |m c| small against 2^24 (r is up to 2^-24 of it, and is an
// exponent), so the running maximum starts at the floor F = -2^k with |F c| in
// (2^19, 2^20] and logits below F count as F. A row whose maximum is not well
// above F (filled with a type's lowest value, say), or is above -F (infinities
// too), is summed again in the plain form 2^((z - m) c) with the subtraction
// first (plain_slice), where any two finite values work; a row masked throughout
// is told by its maximum, and not read again.
// A NaN makes s a NaN, and so does +inf, as exp(z - max) does.
#pragma once

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/drafthead.h"
#include "dh_common.cuh"
#include "dh_internal.h"

namespace dh {
namespace rows {

constexpr int kMaxCluster = 8;   // CTAs per row
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;

// ------------------------------------------------------------ element types --

template <class T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
    static constexpr int kVec = 8;
    __device__ static float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    __device__ static void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    // The largest of U vectors' logits (a NaN is passed over).
    template <int U> __device__ static float max_of(const uint4 (&w)[U]) {
        uint32_t m = max2(max2(w[0].x, w[0].y), max2(w[0].z, w[0].w));
#pragma unroll
        for (int u = 1; u < U; ++u) m = max2(max2(m, max2(w[u].x, w[u].y)), max2(w[u].z, w[u].w));
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // Logits below the floor raised to it; a NaN stays.
    __device__ static uint32_t raise2(uint32_t a, uint32_t f) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(f));
        return r;
    }
    __device__ static void raise(uint4& w, uint32_t f) {
        w = make_uint4(raise2(w.x, f), raise2(w.y, f), raise2(w.z, f), raise2(w.w, f));
    }
    __device__ static uint32_t pack2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
    __device__ static __nv_bfloat16 store(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Elem<__half> {
    static constexpr int kVec = 8;
    __device__ static float load(const __half* p) { return __half2float(*p); }
    __device__ static void unpack(const uint4& v, float (&f)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = f16lo(w[i]);
            f[2 * i + 1] = f16hi(w[i]);
        }
    }
    // The largest of U vectors' logits (a NaN is passed over).
    template <int U> __device__ static float max_of(const uint4 (&w)[U]) {
        uint32_t m = max2(max2(w[0].x, w[0].y), max2(w[0].z, w[0].w));
#pragma unroll
        for (int u = 1; u < U; ++u) m = max2(max2(m, max2(w[u].x, w[u].y)), max2(w[u].z, w[u].w));
        return fmaxf(f16lo(m), f16hi(m));
    }
    __device__ static uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // Logits below the floor raised to it; a NaN stays.
    __device__ static uint32_t raise2(uint32_t a, uint32_t f) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(f));
        return r;
    }
    __device__ static void raise(uint4& w, uint32_t f) {
        w = make_uint4(raise2(w.x, f), raise2(w.y, f), raise2(w.z, f), raise2(w.w, f));
    }
    __device__ static uint32_t pack2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static uint4 pack(const float (&f)[8]) {
        return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
    __device__ static __half store(float x) { return __float2half_rn(x); }
};
template <> struct Elem<float> {
    static constexpr int kVec = 4;
    __device__ static float load(const float* p) { return *p; }
    __device__ static void unpack(const uint4& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    template <int U> __device__ static float max_of(const uint4 (&w)[U]) {
        float m = fmaxf(fmaxf(f(w[0].x), f(w[0].y)), fmaxf(f(w[0].z), f(w[0].w)));
#pragma unroll
        for (int u = 1; u < U; ++u) m = fmaxf(fmaxf(m, fmaxf(f(w[u].x), f(w[u].y))), fmaxf(f(w[u].z), f(w[u].w)));
        return m;
    }
    __device__ static float f(uint32_t u) { return __uint_as_float(u); }
    __device__ static uint32_t raise1(uint32_t a, uint32_t floor) {
        float r1;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r1) : "f"(f(a)), "f"(f(floor)));
        return __float_as_uint(r1);
    }
    __device__ static void raise(uint4& w, uint32_t floor) {
        w = make_uint4(raise1(w.x, floor), raise1(w.y, floor), raise1(w.z, floor), raise1(w.w, floor));
    }
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ static float store(float x) { return x; }
};

// 16 elements at p (alignment of the element type only when !VEC), as floats.
template <class T, bool VEC>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
    if constexpr (VEC) {
        constexpr int kVec = Elem<T>::kVec;
#pragma unroll
        for (int i = 0; i < 16 / kVec; ++i)
            Elem<T>::unpack(*reinterpret_cast<const uint4*>(p + i * kVec), reinterpret_cast<float(&)[kVec]>(x[i * kVec]));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = Elem<T>::load(p + i);
    }
}

// 16 bytes whose elements are all -inf (what a lane past the slice holds).
template <class T> __device__ __forceinline__ uint4 neg_inf_vec();
template <> __device__ __forceinline__ uint4 neg_inf_vec<float>() {
    const uint32_t w = 0xFF800000u;
    return make_uint4(w, w, w, w);
}
template <> __device__ __forceinline__ uint4 neg_inf_vec<__nv_bfloat16>() {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
}
template <> __device__ __forceinline__ uint4 neg_inf_vec<__half>() {
    return make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
}

// ------------------------------------------------------------------- slices --

// A row of C elements at z: `head` elements up to the first 16-byte boundary,
// `nvec` whole 16-byte vectors, the rest. CTA `rank` of the row's cluster owns
// the vectors [v0, v1) and, in index order, the elements [lo, hi): the first
// CTA takes the head too and the last one the tail, so that slices are
// contiguous ranges of columns. A cluster has 2^lg CTAs.
struct Slice {
    int head;       // elements before the first vector of the row
    int v0, v1;     // vectors of this CTA
    int lo, hi;     // columns of this CTA
    int tail0;      // first column after the row's vectors
};

template <class T>
__device__ __forceinline__ Slice make_slice(const T* z, int C, unsigned rank, unsigned lg) {
    constexpr int kVec = Elem<T>::kVec;
    Slice s;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    s.head = mis ? kVec - mis : 0;
    if (s.head > C) s.head = C;
    const int nvec = (C - s.head) / kVec;
    s.v0 = static_cast<int>((static_cast<long long>(nvec) * rank) >> lg);
    s.v1 = static_cast<int>((static_cast<long long>(nvec) * (rank + 1)) >> lg);
    s.tail0 = s.head + nvec * kVec;
    s.lo = rank == 0 ? 0 : s.head + s.v0 * kVec;
    s.hi = rank + 1 == (1u << lg) ? C : s.head + s.v1 * kVec;
    return s;
}

// The column of this thread's single element among those outside the vectors
// (the head in the first CTA, the tail in the last one), or -1. At most 7 + 7.
__device__ __forceinline__ int edge_column(const Slice& s, int C, unsigned rank, unsigned ncta) {
    const int t = static_cast<int>(threadIdx.x);
    const int nh = rank == 0 ? s.head : 0;
    if (t < nh) return t;
    if (rank == ncta - 1 && t - nh < C - s.tail0) return s.tail0 + t - nh;
    return -1;
}

// -------------------------------------------------------- softmax statistics --

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two 32-bit floats at a time.
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct Stat {
    float m, s, s1;
};

// mc of the maximum m, rounded on its own (never fused into a multiply-add), so
// that every use of it is the same number; and r = m c - mc.
__device__ __forceinline__ float shift_of(float m, float c) { return __fmul_rn(m, c); }
__device__ __forceinline__ float shift_rest(float m, float c) { return fmaf(m, c, -shift_of(m, c)); }

// Move the sums of st to the maximum m >= st.m.
template <bool ENTROPY>
__device__ __forceinline__ void stat_shift(Stat& st, float m, float c) {
    const float D = shift_of(st.m, c) - shift_of(m, c), a = ex2(D);
    if (ENTROPY) st.s1 = a * fmaf(D, st.s, st.s1);
    st.s *= a;
    st.m = m;
}

template <bool ENTROPY>
__device__ __forceinline__ Stat stat_join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    stat_shift<ENTROPY>(a, m, c);
    stat_shift<ENTROPY>(b, m, c);
    return Stat{m, a.s + b.s, a.s1 + b.s1};
}

// Add U vectors to st (st.m >= floor throughout): one shift of the sums, then
// a multiply-add, an exponential and an addition per logit, all but the
// exponential on pairs (with the entropy, another multiply-add; there the logits
// are raised to the floor first, so that a zero never meets an infinite
// exponent). The maximum is taken on packed pairs of 16-bit logits; `top` is the
// thread's largest logit itself, below the floor too (-inf: none).
template <class T, bool ENTROPY, int U>
__device__ __forceinline__ void stat_add(Stat& st, float& top, uint4 (&w)[U], float c, uint32_t floor2) {
    constexpr int kVec = Elem<T>::kVec;
    top = fmaxf(top, Elem<T>::template max_of<U>(w));
    const float m = fmaxf(st.m, top);
    if (ENTROPY) {
#pragma unroll
        for (int u = 0; u < U; ++u) Elem<T>::raise(w[u], floor2);
    }
    stat_shift<ENTROPY>(st, m, c);
    const float mc = shift_of(m, c);
    const uint64_t c2 = pack_f32x2(c, c), nmc2 = pack_f32x2(-mc, -mc);
    uint64_t s[2] = {0, 0}, s1[2] = {0, 0};   // of these vectors alone: few roundings at the size of the running sum
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float z[kVec];
        Elem<T>::unpack(w[u], z);
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
            const uint64_t x = fma_f32x2(pack_f32x2(z[i], z[i + 1]), c2, nmc2);
            float x0, x1;
            unpack_f32x2(x, x0, x1);
            const uint64_t e = pack_f32x2(ex2(x0), ex2(x1));
            s[(i >> 1) & 1] = add_f32x2(s[(i >> 1) & 1], e);
            if (ENTROPY) s1[(i >> 1) & 1] = fma_f32x2(e, x, s1[(i >> 1) & 1]);
        }
    }
    float lo, hi;
    unpack_f32x2(add_f32x2(s[0], s[1]), lo, hi);
    st.s += lo + hi;
    if (ENTROPY) {
        unpack_f32x2(add_f32x2(s1[0], s1[1]), lo, hi);
        st.s1 += lo + hi;
    }
}

template <bool ENTROPY>
__device__ __forceinline__ void stat_add1(Stat& st, float z, float c, float floor) {
    stat_shift<ENTROPY>(st, fmaxf(st.m, z), c);
    const float x = fmaf(z < floor ? floor : z, c, -shift_of(st.m, c)), e = ex2(x);   // a NaN stays
    st.s += e;
    if (ENTROPY) st.s1 = fmaf(e, x, st.s1);
}

// True if the sums around the maximum m hold (see the top of this file).
__device__ __forceinline__ bool stat_fits(float m, float c, float floor) {
    return (m - floor) * c > 200.0f && m <= -floor;
}

// The plain form, for any values: s = sum 2^((z - m) c) with the subtraction
// first. A difference is capped at 200, where the power is 0 in 32 bits anyway,
// so that an infinite one never meets a zero sum.
template <bool ENTROPY>
__device__ __forceinline__ void plain_shift(Stat& st, float m, float c) {
    const float D = fminf((m - st.m) * c, 200.0f), a = ex2(-D);
    if (ENTROPY) st.s1 = a * fmaf(-D, st.s, st.s1);
    st.s *= a;
    st.m = m;
}
template <bool ENTROPY>
__device__ __forceinline__ Stat plain_join(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m);
    plain_shift<ENTROPY>(a, m, c);
    plain_shift<ENTROPY>(b, m, c);
    return Stat{m, a.s + b.s, a.s1 + b.s1};
}
template <bool ENTROPY>
__device__ __forceinline__ void plain_add1(Stat& st, float z, float c) {
    plain_shift<ENTROPY>(st, fmaxf(st.m, z), c);
    const float x = (z - st.m) * c, e = ex2(x);
    st.s += e;
    if (ENTROPY) st.s1 = fmaf(e, fmaxf(x, -200.0f), st.s1);
}

// U vectors in the plain form.
template <class T, bool ENTROPY, int U>
__device__ __forceinline__ void plain_add(Stat& st, const uint4 (&w)[U], float c) {
    constexpr int kVec = Elem<T>::kVec;
    plain_shift<ENTROPY>(st, fmaxf(st.m, Elem<T>::template max_of<U>(w)), c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float z[kVec];
        Elem<T>::unpack(w[u], z);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const float x = (z[i] - st.m) * c, e = ex2(x);
            st.s += e;
            if (ENTROPY) st.s1 = fmaf(e, fmaxf(x, -200.0f), st.s1);
        }
    }
}

template <bool ENTROPY, bool PLAIN>
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    return PLAIN ? plain_join<ENTROPY>(a, b, c) : stat_join<ENTROPY>(a, b, c);
}

// The largest of a warp's values (none of them NaN), in every lane.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// Statistics of a warp's lanes joined: one common maximum, then plain sums.
template <bool ENTROPY, bool PLAIN>
__device__ __forceinline__ Stat stat_warp(Stat st, float c) {
    const float m = warp_max(st.m);
    if (PLAIN) plain_shift<ENTROPY>(st, m, c);
    else stat_shift<ENTROPY>(st, m, c);
    st.s = warp_sum(st.s);
    if (ENTROPY) st.s1 = warp_sum(st.s1);
    return st;
}

// Statistics of the CTA's NW warps: each warp leaves its own in buf, and after a
// barrier of the caller's any warp joins them all (the same in every lane).
__device__ __forceinline__ void stat_leave(const Stat& st, float (*buf)[3]) {
    if ((threadIdx.x & 31) == 0) {
        float* b = buf[threadIdx.x >> 5];
        b[0] = st.m;
        b[1] = st.s;
        b[2] = st.s1;
    }
}
template <bool ENTROPY, bool PLAIN>
__device__ __forceinline__ Stat stat_gather(int nw, float c, const float (*buf)[3], float idle_m) {
    const int l = threadIdx.x & 31;
    Stat st = {idle_m, 0.0f, 0.0f};
    if (l < nw) st = Stat{buf[l][0], buf[l][1], buf[l][2]};
    return stat_warp<ENTROPY, PLAIN>(st, c);
}

// Cluster barrier that orders shared-memory writes, remote ones included.
__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait_acquire() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long x) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(addr), "l"(x) : "memory");
}

// Statistics of the row from those of its cluster's CTAs, joined in rank order
// (the same in every CTA). `all`: an entry per rank, which the peers write; a
// caller uses another one in its next call. The peers are known to run (the
// caller passed a cluster barrier before).
template <bool ENTROPY, bool PLAIN>
__device__ __forceinline__ Stat stat_cluster(Stat st, float c, float (*all)[3], unsigned rank, unsigned ncta) {
    if (ncta == 1) return st;
    if (threadIdx.x < ncta) {
        const uint32_t at = cluster_map(&all[rank][0], threadIdx.x);
        st_cluster_f32(at, st.m);
        st_cluster_f32(at + 4, st.s);
        st_cluster_f32(at + 8, st.s1);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    Stat r = Stat{all[0][0], all[0][1], all[0][2]};
    for (unsigned i = 1; i < ncta; ++i) r = join<ENTROPY, PLAIN>(r, Stat{all[i][0], all[i][1], all[i][2]}, c);
    return r;
}

// Column of an id: through row_of (target id -> row, -1 when not kept) when it
// is given; -1 for an id outside the vocabulary or a column outside [0, C).
__device__ __forceinline__ int column_of(int id, const int32_t* row_of, int V, int C) {
    if (row_of != nullptr) {
        if (id < 0 || id >= V) return -1;
        id = __ldg(row_of + id);
    }
    return id >= 0 && id < C ? id : -1;
}

// The largest of the threads' `top` over the row (every thread of its cluster calls
// this; rare). buf and all as for the row's statistics.
template <int NT>
__device__ __noinline__ float row_top(float top, float (*buf)[3], float (*all)[3], unsigned rank, unsigned ncta) {
    const float w = warp_max(top);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5][0] = w;
    __syncthreads();
    float m = warp_max(buf[(threadIdx.x & 31) % (NT / 32)][0]);
    __syncthreads();
    if (ncta > 1) {
        if (threadIdx.x < ncta) st_cluster_f32(cluster_map(&all[rank][0], threadIdx.x), m);
        cluster_arrive_release();
        cluster_wait_acquire();
        for (unsigned i = 0; i < ncta; ++i) m = fmaxf(m, all[i][0]);
        cluster_arrive_release();   // read before the entries are written again
        cluster_wait_acquire();
    }
    return m;
}

// The statistics of a CTA's slice in the plain form, from global memory, U vectors at a time.
template <class T, bool ENTROPY, int NT, int U>
__device__ __forceinline__ Stat plain_slice_of(const T* z, const Slice& sl, float ze, float c, float (*buf)[3]) {
    constexpr int kVec = Elem<T>::kVec;
    Stat st = {-FLT_MAX, 0.0f, 0.0f};
    plain_add1<ENTROPY>(st, ze, c);
#pragma unroll 1
    for (int v0 = sl.v0 + threadIdx.x; v0 < sl.v1; v0 += U * NT) {
        uint4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = v0 + u * NT < sl.v1 ? *reinterpret_cast<const uint4*>(z + sl.head + static_cast<size_t>(v0 + u * NT) * kVec)
                                       : neg_inf_vec<T>();
        plain_add<T, ENTROPY, U>(st, w, c);
    }
    st = stat_warp<ENTROPY, true>(st, c);
    stat_leave(st, buf);
    __syncthreads();
    return stat_gather<ENTROPY, true>(NT / 32, c, buf, -FLT_MAX);
}

// The same out of line, for rows that stat_fits() refuses and that are not masked
// throughout (rare).
template <class T, bool ENTROPY, int NT>
__device__ __noinline__ Stat plain_slice(const T* z, const Slice& sl, float ze, float c, float (*buf)[3]) {
    return plain_slice_of<T, ENTROPY, NT, 4>(z, sl, ze, c, buf);
}

// ---------------------------------------------------------------- streaming --

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// The rows of a persistent cluster, streamed through shared memory. Every
// thread copies its own vectors (vector i of thread a of a slice is v0 + a + i NT)
// into its own column of the ring and reads only those back, so the stream
// needs no barrier: a batch of U vectors is one cp.async group, P batches are in
// flight, and the fetching runs on into the next rows while a row's ends are
// worked on. Every step commits exactly one group (an empty one where nothing
// is left to fetch), so the batch of a step is always the P-th last group.
// `passes`: how often each row is streamed before the next one.
template <class T, int NT, int U, int P>
struct Stream {
    static constexpr int kBytes = P * U * NT * 16, kSlot = U * NT * 16;
    static constexpr int kVec = Elem<T>::kVec;
    const T* z;
    long long ld;
    int M, C, passes;
    unsigned rank, lg;
    int stride;          // rows between two of this cluster
    bool alike;          // rows share their offset from a 16-byte boundary, so their slices are alike
    int row;             // fetch position: row, batch
    int batch, batches, left;
    int after;           // vectors of the slice from this thread's first vector on
    const uint4* at;     // this thread's first vector of the row
    const uint4* cur;    // and of the next batch
    uint32_t base, slot; // this thread's column of the ring; offset of the next fetch

    __device__ static __forceinline__ int batches_of(const Slice& s) { return (s.v1 - s.v0 + NT * U - 1) / (NT * U); }

    __device__ __forceinline__ void open_row(bool first) {
        if (row >= M) return;
        if (first || !alike) {
            const T* p = z + static_cast<size_t>(row) * ld;
            const Slice sl = make_slice(p, C, rank, lg);
            batches = batches_of(sl);
            after = sl.v1 - sl.v0 - static_cast<int>(threadIdx.x);
            at = reinterpret_cast<const uint4*>(p + sl.head) + sl.v0 + threadIdx.x;
        } else {
            at = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(at) + static_cast<size_t>(stride) * ld);
        }
        batch = 0;
        cur = at;
        left = passes * batches;
    }

    __device__ __forceinline__ void start(const T* z_, long long ld_, int M_, int C_, unsigned rank_, unsigned lg_, int row0,
                                          int stride_, void* ring, int passes_ = 1) {
        z = z_;
        ld = ld_;
        M = M_;
        C = C_;
        rank = rank_;
        lg = lg_;
        row = row0;
        stride = stride_;
        passes = passes_;
        alike = (ld * static_cast<long long>(sizeof(T))) % 16 == 0;
        base = smem_u32(ring) + threadIdx.x * 16;
        slot = 0;
        left = 0;
        open_row(true);
#pragma unroll 1
        for (int i = 0; i < P; ++i) fetch();
    }
    __device__ static __forceinline__ uint32_t next(uint32_t s) { return s + kSlot == kBytes ? 0 : s + kSlot; }

    __device__ __forceinline__ void copy(int u) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(base + slot + u * (NT * 16)), "l"(cur + u * NT) : "memory");
    }

    // Fetch the next batch into the ring's next slot (whose last batch this thread has read).
    __device__ __forceinline__ void fetch() {
        while (left == 0 && row < M) {
            row += stride;
            open_row(false);
        }
        if (row < M) {
            if (batch + 1 < batches) {
#pragma unroll
                for (int u = 0; u < U; ++u) copy(u);
            } else {
                const int n = after - batch * (NT * U);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u * NT < n) copy(u);
            }
            cur += NT * U;
            if (++batch == batches) {
                batch = 0;
                cur = at;
            }
            --left;
        }
        cp_async_commit();
        slot = next(slot);
    }

    // The vectors of the batch at offset s (batch b of slice q); -inf past the slice's end.
    __device__ __forceinline__ void read(uint32_t s, const Slice& q, int b, uint4 (&w)[U]) const {
#pragma unroll
        for (int u = 0; u < U; ++u)
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[u].x), "=r"(w[u].y), "=r"(w[u].z), "=r"(w[u].w) : "r"(base + s + u * (NT * 16)) : "memory");
        if (q.v0 + (b + 1) * (NT * U) > q.v1) {
            const int n = q.v1 - q.v0 - b * (NT * U) - static_cast<int>(threadIdx.x);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (u * NT >= n) w[u] = neg_inf_vec<T>();
        }
    }
};

// The ids of this thread's entry, fetched ahead of their rows, so that the chain
// id -> column -> logit costs a row one load's latency at most and no load is
// waited for in the call that issues it. Call take() once per row, in order.
// `entry`: the entry of a row that this thread looks after (a warp without entries
// skips it all).
struct IdAhead {
    const int32_t* ids;
    const int32_t* row_of;
    int n, V, C, M, stride, entry;
    int ahead;      // the id in the row after the next one
    int id, col;    // the id in the next row, and what row_of holds for it

    __device__ __forceinline__ bool idle() const { return (entry & ~31) >= n; }   // a warp's lanes alike
    __device__ __forceinline__ int load(int row) const {
        return row < M && entry < n ? __ldg(ids + static_cast<size_t>(row) * n + entry) : -1;
    }
    __device__ __forceinline__ void look(int of) {
        id = of;
        col = row_of != nullptr ? __ldg(row_of + min(max(of, 0), V - 1)) : of;
    }
    __device__ __forceinline__ void start(int row) {
        if (idle()) return;
        look(load(row));
        ahead = load(row + stride);
    }
    // The column in `row` (-1: none, or no entry for this thread).
    __device__ __forceinline__ int take(int row) {
        if (idle()) return -1;
        const int now = (row_of == nullptr || (id >= 0 && id < V)) && col >= 0 && col < C ? col : -1;
        look(ahead);
        ahead = load(row + 2 * stride);
        return now;
    }
};

// ------------------------------------------------------------------- launch --

// The floor of the statistics: -2^k with c 2^k in (2^19, 2^20], as the type can
// hold it; 0 (no row fits, all are summed in the plain form) where it cannot.
// `floor2`: its bits, twice for a 16-bit type.
inline void set_floor(int type, float c, float& floor, uint32_t& floor2) {
    int e;
    frexpf(c, &e);   // c in [2^(e-1), 2^e)
    int k = 20 - e;
    if (type == DH_T_F16 && k > 15) k = 15;
    if (k > 126) k = 126;
    floor = k < (type == DH_T_F16 ? -14 : -126) ? 0.0f : -ldexpf(1.0f, k);
    uint32_t bits;
    std::memcpy(&bits, &floor, 4);
    if (type == DH_T_BF16) bits = bits >> 16 | (bits & 0xFFFF0000u);
    if (type == DH_T_F16) {   // -2^k, normal
        const uint32_t h = floor == 0.0f ? 0u : 0x8000u | static_cast<uint32_t>(k + 15) << 10;
        bits = h | h << 16;
    }
    floor2 = bits;
}

// What a launch of KERNEL needs to know of a device, found on its first call
// there: clusters of 2^lg CTAs that fit the GPU at once.
struct RowLaunch {
    int fit[4];
};

template <class A, void (*KERNEL)(A)>
static cudaError_t row_launch_setup(int threads, int smem, RowLaunch& out) {
    cudaError_t e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    for (unsigned lg = 0; e == cudaSuccess && lg < 4; ++lg) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1u << lg);
        cfg.blockDim = dim3(static_cast<unsigned>(threads));
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 1u << lg;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&out.fit[lg], KERNEL, &cfg);
    }
    return e;
}

// Costs of a row beyond reading it, in bytes read in the same time: `fixed` for
// its ends, `exchange` more where a cluster shares it; `twice`: the row is streamed
// twice, from L2 the second time if the rows in work fit there.
struct RowCost {
    long long fixed, exchange;
    bool twice;
};
constexpr long long kRowsInL2 = 64ll << 20;   // of the 129 MB, beside what is written

// Launch a persistent kernel over M rows. CTAs per row, by the time of the
// longest-working CTA: rounds of rows that a cluster takes times its CTA's share
// of a row (half as much again for a row streamed twice that does not stay in L2)
// and its costs. Few long rows are so split over up to 8 CTAs (16 rows of 248,320
// f32, log-probabilities: 13.5 us), long rows streamed twice over as many as keep
// them in L2 (573 rows of 228,680 f32, loss and gradient: 203 us over eight CTAs, 260 unsplit;
// 1,200 of 128,000 bf16: 123 over two, 142), and rows that fill the GPU or are short are not split
// (20 alternatives of 268 rows of 34,166 bf16: 9.9 us unsplit, 32 over clusters
// of four in three rounds; of 4 rows of 2,743 f32: 6.6 unsplit, 10.5 over eight).
template <class A, void (*KERNEL)(A)>
static cudaError_t launch_rows(A a, long long row_bytes, RowCost c, int threads, int smem, cudaStream_t s) {
    constexpr int kDevices = 64;
    static std::atomic<bool> known[kDevices];
    static std::atomic<int> fits[kDevices][4];   // (concurrent first callers store equal values)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        RowLaunch l = {};
        if ((e = row_launch_setup<A, KERNEL>(threads, smem, l)) != cudaSuccess) return e;
        for (int i = 0; i < 4; ++i) fits[dev][i].store(l.fit[i], std::memory_order_relaxed);
        known[dev].store(true, std::memory_order_release);
    }
    RowLaunch fit;
    for (int i = 0; i < 4; ++i) fit.fit[i] = fits[dev][i].load(std::memory_order_relaxed);
    unsigned lg = 0;
    long long best = 0;
    for (unsigned l = 0; l < 4 && fit.fit[l] > 0; ++l) {
        const long long rounds = (a.M + fit.fit[l] - 1) / fit.fit[l];
        const bool spills = c.twice && (a.M < fit.fit[l] ? a.M : fit.fit[l]) * row_bytes > kRowsInL2;
        const long long share = row_bytes >> l;
        const long long cost = rounds * ((spills ? share + share / 2 : share) + c.fixed + (l > 0 ? c.exchange : 0));
        if (l == 0 || cost < best) {
            best = cost;
            lg = l;
        }
    }
    a.lg = lg;
    const int clusters = a.M < fit.fit[lg] ? a.M : fit.fit[lg];
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters) << lg);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 1u << lg;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = lg > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, KERNEL, a);
}

}  // namespace rows
}  // namespace dh
