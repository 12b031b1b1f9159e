// Helpers of the operators on rows of logits (token log-probabilities,
// distillation): element types, a row's split into 16-byte vectors over the
// CTAs of a cluster, and the running softmax statistics.
//
// Statistics of a set of logits z, at temperature t with c = log2(e) / t:
//   m  = max z                       (-FLT_MAX for an empty or all -inf set),
//   s  = sum 2^((z - m) c),
//   s1 = sum 2^((z - m) c) (z - m) c (for the entropy),
// all in 32 bits. Two sets are joined by scaling each one's sums to the common
// maximum: with D = (m' - m) c, s' = 2^-D s and s1' = 2^-D (s1 - D s). D is
// capped at 200, where 2^-D is 0 in 32 bits anyway, so that an infinite D
// never meets a zero sum. The shift z - m is a subtraction of its own (not
// folded into a multiply-add with m c), so that rows of the types' lowest
// values, whose product with c overflows, still sum correctly. A NaN or +inf
// logit makes s a NaN, as exp(z - max) does.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dh_common.cuh"

namespace dh {
namespace rows {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
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
    __device__ static uint4 pack(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ static float store(float x) { return x; }
};

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
// contiguous ranges of columns.
struct Slice {
    int head;       // elements before the first vector of the row
    int v0, v1;     // vectors of this CTA
    int lo, hi;     // columns of this CTA
    int tail0;      // first column after the row's vectors
};

template <class T>
__device__ __forceinline__ Slice make_slice(const T* z, int C, unsigned rank, unsigned ncta) {
    constexpr int kVec = Elem<T>::kVec;
    Slice s;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(T));
    s.head = mis ? kVec - mis : 0;
    if (s.head > C) s.head = C;
    const int nvec = (C - s.head) / kVec;
    s.v0 = static_cast<int>(static_cast<long long>(nvec) * rank / ncta);
    s.v1 = static_cast<int>(static_cast<long long>(nvec) * (rank + 1) / ncta);
    s.tail0 = s.head + nvec * kVec;
    s.lo = rank == 0 ? 0 : s.head + s.v0 * kVec;
    s.hi = rank == ncta - 1 ? C : s.head + s.v1 * kVec;
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

struct Stat {
    float m, s, s1;
};

__device__ __forceinline__ Stat stat_empty() { return Stat{-FLT_MAX, 0.0f, 0.0f}; }

// The sums of st moved to the maximum m >= st.m.
template <bool ENTROPY>
__device__ __forceinline__ void stat_shift(Stat& st, float m, float c) {
    const float D = fminf((m - st.m) * c, 200.0f);
    const float a = ex2(-D);
    if (ENTROPY) st.s1 = a * fmaf(-D, st.s, st.s1);
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

// Add N values (N even) to st: one shift of the sums per call, then two values
// at a time (packed 32-bit arithmetic).
template <bool ENTROPY, int N>
__device__ __forceinline__ void stat_add(Stat& st, const float (&z)[N], float c) {
    float m = st.m;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, z[i]);
    stat_shift<ENTROPY>(st, m, c);
    const uint64_t nm = pack_f32x2(-m, -m), cc = pack_f32x2(c, c);
    uint64_t s = pack_f32x2(st.s, 0.0f), s1 = pack_f32x2(st.s1, 0.0f);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t x = mul_f32x2(add_f32x2(pack_f32x2(z[i], z[i + 1]), nm), cc);
        float x0, x1;
        unpack_f32x2(x, x0, x1);
        const uint64_t e = pack_f32x2(ex2(x0), ex2(x1));
        s = add_f32x2(s, e);
        // a zero term: 2^x is 0 where x is below -200, so x may be replaced there
        if (ENTROPY) s1 = fma_f32x2(e, pack_f32x2(fmaxf(x0, -200.0f), fmaxf(x1, -200.0f)), s1);
    }
    float a, b;
    unpack_f32x2(s, a, b);
    st.s = a + b;
    if (ENTROPY) {
        unpack_f32x2(s1, a, b);
        st.s1 = a + b;
    }
}

template <bool ENTROPY>
__device__ __forceinline__ void stat_add1(Stat& st, float z, float c) {
    const float v[2] = {z, kNegInf};
    stat_add<ENTROPY, 2>(st, v, c);
}

template <bool ENTROPY>
__device__ __forceinline__ Stat stat_warp(Stat st, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
        b.s = __shfl_xor_sync(0xFFFFFFFFu, st.s, o);
        b.s1 = ENTROPY ? __shfl_xor_sync(0xFFFFFFFFu, st.s1, o) : 0.0f;
        st = stat_join<ENTROPY>(st, b, c);
    }
    return st;
}

// Statistics of the whole CTA, the same in every thread. `buf`: kWarps
// entries, free to be written again after the caller's next __syncthreads.
template <bool ENTROPY>
__device__ __forceinline__ Stat stat_block(Stat st, float c, float (*buf)[3]) {
    st = stat_warp<ENTROPY>(st, c);
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    if (l == 0) {
        buf[w][0] = st.m;
        buf[w][1] = st.s;
        buf[w][2] = st.s1;
    }
    __syncthreads();
    Stat r = stat_empty();
    if (l < kWarps) r = Stat{buf[l][0], buf[l][1], buf[l][2]};
    return stat_warp<ENTROPY>(r, c);
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
// (the same in every CTA). `all`: kMaxCluster entries in shared memory that
// the peers write. The caller has arrived on the cluster barrier once (so that
// every peer is known to run); this waits for it and passes the next one.
template <bool ENTROPY>
__device__ __forceinline__ Stat stat_cluster(Stat st, float c, float (*all)[3], unsigned rank, unsigned ncta) {
    if (ncta == 1) return st;
    cluster_wait_acquire();
    if (threadIdx.x < ncta) {
        const uint32_t at = cluster_map(&all[rank][0], threadIdx.x);
        st_cluster_f32(at, st.m);
        st_cluster_f32(at + 4, st.s);
        st_cluster_f32(at + 8, st.s1);
    }
    cluster_arrive_release();
    cluster_wait_acquire();
    Stat r = Stat{all[0][0], all[0][1], all[0][2]};
    for (unsigned i = 1; i < ncta; ++i) r = stat_join<ENTROPY>(r, Stat{all[i][0], all[i][1], all[i][2]}, c);
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

}  // namespace rows
}  // namespace dh
