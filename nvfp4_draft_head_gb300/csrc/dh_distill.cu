// Distillation of the student's logits rows z [M][C] from a teacher's top K
// logits, at temperature t, with row weights w:
//
//   p = softmax(teacher / t) over the row's entries in use, q = softmax(z / t),
//   loss = w t^2 sum_j p_j (log p_j - log q_j),    dz_c = w t (q_c - p_c).
//
// An entry is in use when its id has a column, neither its own logit nor the
// student's is -inf, and the row's weight is not zero; the others leave the
// teacher's distribution, which is normalised over what remains. A row with no
// entry in use has loss 0 and gradient 0. (d(log q_j)/dz_c = (delta_jc - q_c)/t
// and sum p = 1 give the gradient.) Entries that name one column twice add up.
//
// One cluster of 1..8 CTAs per row. Every CTA takes the whole teacher row (one
// entry per thread, its column and the student's logit there fetched before
// the row is streamed), the statistics of its slice as in dh_rows.cuh, and
// writes its slice of the gradient: first w t q everywhere, then, after a
// barrier, the columns of the teacher's entries again with p taken off. The
// sums are joined in a fixed order, so results repeat bit for bit. The gradient
// may be written over the logits: a CTA reads every logit that it needs outside
// its slice before the cluster barrier that precedes the first write.
//
// Bound: HBM. Loss and gradient together read the row twice; the second time
// it comes from L2 (see the launcher).
#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_rows.cuh"

namespace dh {
namespace rows {

constexpr int kUnroll = 4;   // vectors in flight per thread

struct DistillSmem {
    float warp[kWarps][3];
    float teach[kWarps][3];
    float cta[kMaxCluster][3];
    float red[kWarps];
    int col[kThreads];
    float p[kThreads];
};

// Plain (coherent) 16-byte load: the row may be overwritten by this kernel.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ void st_v4(void* p, const uint4& v) {
    asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = 0.0f;
    for (int w = 0; w < kWarps; ++w) r += buf[w];
    return r;
}

// Element i of an array whose type is known at run time.
__device__ __forceinline__ float load_as(const void* p, size_t i, int type) {
    if (type == DH_T_BF16) return Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p) + i);
    if (type == DH_T_F16) return Elem<__half>::load(static_cast<const __half*>(p) + i);
    return static_cast<const float*>(p)[i];
}

template <class T, DistillMode MODE>
__global__ void __launch_bounds__(kThreads, 2) distill_kernel(const DistillArgs a) {
    constexpr int kVec = Elem<T>::kVec;
    constexpr bool kGrad = MODE != kDistillForward, kStats = MODE != kDistillBackward;
    __shared__ DistillSmem sm;
    const unsigned rank = cluster_ctarank(), ncta = a.ncta;
    const int row = blockIdx.x / ncta, tid = threadIdx.x;
    if (ncta > 1) cluster_arrive_release();
    const T* z = static_cast<const T*>(a.z) + static_cast<size_t>(row) * a.ld;
    const Slice sl = make_slice(z, a.C, rank, ncta);
    const int edge = edge_column(sl, a.C, rank, ncta);
    const float c = a.inv_t * kLog2e;
    const float w = a.weight != nullptr ? __ldg(a.weight + row) : 1.0f;

    // the teacher's entry of this thread
    int col = -1;
    float t = kNegInf, zt = kNegInf;
    if (tid < a.K && w != 0.0f) {
        const size_t at = static_cast<size_t>(row) * a.K + tid;
        col = column_of(a.ids[at], a.row_of, a.V, a.C);
        t = load_as(a.val, at, a.val_type);
        if (col >= 0) zt = Elem<T>::load(z + col);
    }
    const bool used = col >= 0 && t != kNegInf && zt != kNegInf;
    const bool some = __syncthreads_or(used);

    Stat all = stat_empty();
    if (kStats && (some || MODE == kDistillForward)) {
        Stat st = stat_empty();
        for (int v0 = sl.v0 + tid; v0 < sl.v1; v0 += kUnroll * kThreads) {
            uint4 b[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int v = v0 + u * kThreads;
                b[u] = v < sl.v1 ? ld_v4(z + sl.head + static_cast<size_t>(v) * kVec) : neg_inf_vec<T>();
            }
            float x[kUnroll * kVec];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) Elem<T>::unpack(b[u], reinterpret_cast<float(&)[kVec]>(x[u * kVec]));
            stat_add<false>(st, x, c);
        }
        if (edge >= 0) stat_add1<false>(st, Elem<T>::load(z + edge), c);
        all = stat_block<false>(st, c, sm.warp);
    }
    // every CTA of the cluster takes the same path here: `some` is the row's
    if (kStats) {
        all = stat_cluster<false>(all, c, sm.cta, rank, ncta);
    } else if (ncta > 1) {
        cluster_wait_acquire();
        cluster_arrive_release();   // no CTA writes its slice before all have read theirs from it
        cluster_wait_acquire();
    }

    // the teacher's distribution over the entries in use
    float p = 0.0f, logp = 0.0f;
    if (some) {
        Stat ts = stat_empty();
        if (used) stat_add1<false>(ts, t, c);
        ts = stat_block<false>(ts, c, sm.teach);
        if (used) {
            const float d = (t - ts.m) * a.inv_t;
            p = expf(d) / ts.s;
            logp = d - logf(ts.s);
        }
    }

    if (kStats && rank == 0) {
        const float ln_s = logf(all.s);
        if (MODE == kDistillForward && tid == 0 && a.lse != nullptr)
            a.lse[row] = all.s == 0.0f ? kNegInf : all.m * a.inv_t + ln_s;
        float loss = 0.0f;
        if (some) {
            // an entry whose probability underflows adds nothing
            const float logq = (zt - all.m) * a.inv_t - ln_s;
            loss = block_sum(used && p != 0.0f ? p * (logp - logq) : 0.0f, sm.red);
        }
        if (tid == 0) a.loss[row] = some ? w * a.t * a.t * loss : 0.0f;
    }
    if (!kGrad) return;

    // dz = scale * 2^((z - m) c) with scale = w t / S; from a kept normaliser, w t e^(z / t - lse)
    const float wt = w * a.t;
    const float shift = kStats ? all.m : a.lse_in[row];
    const float scale = !some ? 0.0f : kStats ? wt / all.s : wt;
    const auto wtq = [&](float x) {
        return scale * ex2(kStats ? (x - shift) * c : fmaf(x, a.inv_t, -shift) * kLog2e);
    };
    T* dz = static_cast<T*>(a.dz) + static_cast<size_t>(row) * a.ld_dz;
    const bool vec_out = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15u) == 0;
    for (int v0 = sl.v0 + tid; v0 < sl.v1; v0 += kUnroll * kThreads) {
        uint4 b[kUnroll];
        if (some) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int v = v0 + u * kThreads;
                b[u] = v < sl.v1 ? ld_v4(z + sl.head + static_cast<size_t>(v) * kVec) : neg_inf_vec<T>();
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * kThreads;
            if (v >= sl.v1) break;
            float x[kVec];
            if (some) {
                Elem<T>::unpack(b[u], x);
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[j] = wtq(x[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[j] = 0.0f;
            }
            T* out = dz + sl.head + static_cast<size_t>(v) * kVec;
            if (vec_out) {
                st_v4(out, Elem<T>::pack(x));
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) out[j] = Elem<T>::store(x[j]);
            }
        }
    }
    if (edge >= 0) dz[edge] = Elem<T>::store(some ? wtq(Elem<T>::load(z + edge)) : 0.0f);
    if (!some) return;

    // the teacher's columns of this slice: one thread per column, the first entry that names it
    if (tid < a.K) {
        sm.col[tid] = used ? col : -1;
        sm.p[tid] = p;
    }
    __syncthreads();   // also orders the stores above before those below
    if (used && col >= sl.lo && col < sl.hi) {
        float sum = 0.0f;
        bool first = true;
        for (int j = 0; j < a.K; ++j) {
            if (sm.col[j] != col) continue;
            first = first && j >= tid;
            sum += sm.p[j];
        }
        if (first) dz[col] = Elem<T>::store(wtq(zt) - wt * sum);
    }
}

template <class T, DistillMode MODE>
static cudaError_t launch(const DistillArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M) * a.ncta);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.ncta;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, MODE>, a);
}

template <class T>
static cudaError_t launch_mode(const DistillArgs& a, DistillMode mode, cudaStream_t s) {
    switch (mode) {
        case kDistillForward: return launch<T, kDistillForward>(a, s);
        case kDistillBoth: return launch<T, kDistillBoth>(a, s);
        default: return launch<T, kDistillBackward>(a, s);
    }
}

}  // namespace rows

cudaError_t launch_distill(DistillArgs a, int type, DistillMode mode, cudaStream_t s) {
    using namespace rows;
    a.ncta = static_cast<unsigned>(cluster_size(a.M, static_cast<long long>(a.C) * (type == DH_T_F32 ? 4 : 2)));
    switch (type) {
        case DH_T_BF16: return launch_mode<__nv_bfloat16>(a, mode, s);
        case DH_T_F16: return launch_mode<__half>(a, mode, s);
        default: return launch_mode<float>(a, mode, s);
    }
}

}  // namespace dh
