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
// Persistent clusters of 1..8 CTAs take the rows in turn. Every CTA takes the
// whole teacher row (one entry per thread, its column looked up a row ahead and
// the student's logit there fetched before the row is worked on), the statistics
// of its slice as in dh_rows.cuh, and writes its slice of the gradient: first
// w t q everywhere, then the columns of the teacher's entries again with p taken
// off (after the next row's barrier, so that a row costs one barrier). The sums are
// joined in a fixed order, so results repeat bit for bit. The gradient may be
// written over the logits: a CTA reads every logit that it needs outside its slice
// before the cluster barrier that precedes the first write.
//
// Loss and gradient together stream every row twice; the second time it comes
// from L2, where the rows in work (three per SM) fit.
//
// Bound: latency at three CTAs per SM (issue 57 of 100 cycles, loads and the barriers of
// a row's ends the largest stalls), near HBM. Loss and gradient of 4,096 rows of 64,026
// bf16: 202 us, 5.2 of the measured 6.8 TB/s (155 us); 14 instructions per 32 logits and
// 5,600 a row. The gradient alone, 256 rows of 248,320 f32: 84 us (75), the loss alone,
// 1,021 rows of 64,026 bf16, a tenth of them masked throughout: 30 us (19). Three CTAs
// of 256 threads per SM (512 threads twice: 244 us; 256 threads twice 206, four
// times 240). A row held whole in shared memory between its two passes, one CTA of
// 512 or 1,024 threads per SM: 265 to 360 us, the ends of a row then run alone.
#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_rows.cuh"

namespace dh {
namespace rows {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;    // vectors per batch and thread
constexpr int kDepth = 2;     // batches in flight: 32 KB per CTA
constexpr int kPerSm = 3;     // CTAs per SM
// A kept normaliser is rounded to 32 bits, and e^(z / t - lse) carries that rounding, half the
// spacing of such numbers: 3e-5 up to this limit. Rows farther from zero (at a type's lowest
// value throughout, say, where the logarithm of the sum is lost altogether) are summed again from
// their logits: 256 rows of 248,320 f32, all of them so, 127 us against 86.
constexpr float kLseLimit = 1024.0f;

struct DistillSmem {
    float warp[2][kWarps][3];
    float plain[kWarps][3];
    float teach[2][kWarps][3];
    float cta[2][kMaxCluster][3];
    float cta_plain[kMaxCluster][3];
    int used[2][kWarps];
    float red[2][kWarps];
    alignas(16) int col[2][DH_MAX_TEACHER];
    float p[2][DH_MAX_TEACHER];
};

__device__ __forceinline__ void st_v4(void* p, const uint4& v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A vector of gradients, element by element where the rows of the gradient lie at
// another offset from a 16-byte boundary than the logits'.
template <class T>
__device__ __forceinline__ void store_vec(T* p, const uint4& g, bool whole) {
    if (whole) {
        st_v4(p, g);
    } else {
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<uint32_t*>(p)[i] = w[i];
            } else {
                reinterpret_cast<uint16_t*>(p)[2 * i] = static_cast<uint16_t>(w[i]);
                reinterpret_cast<uint16_t*>(p)[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
            }
        }
    }
}

// Element i of an array whose type is known at run time.
__device__ __forceinline__ float load_as(const void* p, size_t i, int type) {
    if (type == DH_T_BF16) return Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p) + i);
    if (type == DH_T_F16) return Elem<__half>::load(static_cast<const __half*>(p) + i);
    return static_cast<const float*>(p)[i];
}

// E: teacher entries per thread.
template <class T, DistillMode MODE, int E>
__global__ void __launch_bounds__(kThreads, kPerSm) distill_kernel(const DistillArgs a) {
    using St = Stream<T, kThreads, kUnroll, kDepth>;
    constexpr int kVec = Elem<T>::kVec;
    constexpr bool kGrad = MODE != kDistillForward, kStats = MODE != kDistillBackward;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ DistillSmem sm;
    const unsigned lg = a.lg, ncta = 1u << lg, rank = ncta > 1 ? cluster_ctarank() : 0u;
    const int first = blockIdx.x >> lg, stride = gridDim.x >> lg, tid = threadIdx.x, warp = tid >> 5;
    const int nt = min((a.K + 31) >> 5, kWarps);   // warps with teacher entries
    const bool teacher = warp < nt;
    static_assert(DH_MAX_TEACHER <= 2 * kThreads, "at most two teacher entries per thread");
    const float c = a.inv_t * kLog2e;
    St stream;
    stream.start(static_cast<const T*>(a.z), a.ld, a.M, a.C, rank, lg, first, stride, ring, MODE == kDistillBoth ? 2 : 1);
    IdAhead ahead[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ahead[e] = {a.ids, a.row_of, a.K, a.V, a.C, a.M, stride, tid + e * kThreads, -1, -1, -1};
        ahead[e].start(first);
    }
    if (ncta > 1) {   // every peer runs before its shared memory is written
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    // the end of a row, after the barrier that follows its gradient
    struct {
        int col[E];       // the teacher's columns of this thread in this slice, or -1
        float base[E];    // w t q there
        float wt;         // w t
        T* dz;
        float loss_w;     // w t^2 (0: no entry in use)
        int row;          // -1: none yet
    } end = {};
    end.row = -1;
#pragma unroll
    for (int e = 0; e < E; ++e) end.col[e] = -1;
    const auto finish = [&](int turn) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (!kGrad || end.col[e] < 0) continue;
            // one thread per column, the first entry that names it
            const int col = end.col[e], entry = tid + e * kThreads;
            float sum = 0.0f;
            bool mine = true;
            const int4* cols = reinterpret_cast<const int4*>(sm.col[turn]);
            for (int j = 0; j < a.K; j += 4) {
                const int4 q = cols[j >> 2];
                if (q.x != col && q.y != col && q.z != col && q.w != col) continue;
                for (int i = j; i < min(j + 4, a.K); ++i) {
                    if (sm.col[turn][i] != col) continue;
                    mine = mine && i >= entry;
                    sum += sm.p[turn][i];
                }
            }
            if (mine) end.dz[col] = Elem<T>::store(end.base[e] - end.wt * sum);
        }
        if (kStats && rank == 0 && tid == 0 && end.row >= 0) {
            float loss = 0.0f;
            if (end.loss_w != 0.0f)
                for (int i = 0; i < nt; ++i) loss += sm.red[turn][i];
            a.loss[end.row] = end.loss_w != 0.0f ? end.loss_w * loss : 0.0f;
        }
    };
    uint32_t slot = 0;
    int turn = 0;
    const T* z = static_cast<const T*>(a.z) + static_cast<size_t>(first) * a.ld;
    T* dz = static_cast<T*>(a.dz) + static_cast<size_t>(first) * a.ld_dz;
    Slice sl = make_slice(z, a.C, rank, lg);
    for (int row = first; row < a.M;
         row += stride, turn ^= 1, z += static_cast<size_t>(stride) * a.ld, dz += static_cast<size_t>(stride) * a.ld_dz) {
        if (!stream.alike) sl = make_slice(z, a.C, rank, lg);
        const int edge = edge_column(sl, a.C, rank, ncta), batches = St::batches_of(sl);
        const float w = a.weight != nullptr ? __ldg(a.weight + row) : 1.0f;
        const float lse = kStats ? 0.0f : __ldg(a.lse_in + row);
        int col[E];
        float t[E], zt[E], ze = kNegInf;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            col[e] = ahead[e].take(row);
            t[e] = zt[e] = kNegInf;
            if (col[e] >= 0) {
                t[e] = load_as(a.val, static_cast<size_t>(row) * a.K + ahead[e].entry, a.val_type);
                zt[e] = Elem<T>::load(z + col[e]);
            }
        }
        if (edge >= 0) ze = Elem<T>::load(z + edge);

        // the statistics of the slice
        Stat all = {a.floor, 0.0f, 0.0f};
        float top = ze;
        if (kStats) {
            for (int b = 0; b < batches; ++b) {
                cp_async_wait<kDepth - 1>();
                uint4 v[kUnroll];
                stream.read(slot, sl, b, v);
                stream.fetch();
                slot = St::next(slot);
                stat_add<T, false, kUnroll>(all, top, v, c, a.floor2);
            }
            if (edge >= 0) stat_add1<false>(all, ze, c, a.floor);
            stat_leave(stat_warp<false, false>(all, c), sm.warp[turn]);
        }
        // the teacher's entries in use, and the sums of their softmax (the student's
        // logits there are in hand before any cluster barrier of this row)
        bool used[E];
#pragma unroll
        for (int e = 0; e < E; ++e) used[e] = col[e] >= 0 && w != 0.0f && t[e] != kNegInf && zt[e] != kNegInf;
        if (teacher) {
            Stat ts = {-FLT_MAX, 0.0f, 0.0f};
            bool any = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (used[e]) plain_add1<false>(ts, t[e], c);
                any = any || used[e];
            }
            any = __any_sync(0xFFFFFFFFu, any);
            stat_leave(stat_warp<false, true>(ts, c), sm.teach[turn]);
            if ((tid & 31) == 0) sm.used[turn][warp] = any;
        }
        __syncthreads();
        finish(turn ^ 1);
        const int l = tid & 31;
        const bool some = __any_sync(0xFFFFFFFFu, l < nt && sm.used[turn][l]);

        // the statistics of the row
        bool plain = false;
        if (kStats) {
            all = stat_gather<false, false>(kWarps, c, sm.warp[turn], a.floor);
            all = stat_cluster<false, false>(all, c, sm.cta[turn], rank, ncta);
            plain = !stat_fits(all.m, c, a.floor);
            if (plain) {   // masked throughout (and no NaN), or summed in the plain form
                if (row_top<kThreads>(top, sm.plain, sm.cta_plain, rank, ncta) == kNegInf && all.s == all.s) {
                    all = Stat{0.0f, 0.0f, 0.0f};
                } else {
                    all = plain_slice<T, false, kThreads>(z, sl, ze, c, sm.plain);
                    all = stat_cluster<false, true>(all, c, sm.cta_plain, rank, ncta);
                }
            }
        } else if (ncta > 1) {   // no CTA writes its slice before all have read theirs from it
            cluster_arrive_release();
            cluster_wait_acquire();
        }

        const float ln_s = kStats ? logf(all.s) - (plain ? 0.0f : shift_rest(all.m, c) * kLn2) : 0.0f;
        if (teacher && some) {
            const Stat ts = stat_gather<false, true>(nt, c, sm.teach[turn], -FLT_MAX);
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float p = 0.0f;
                if (used[e]) {
                    const float d = (t[e] - ts.m) * a.inv_t;
                    p = expf(d) / ts.s;
                    // an entry whose probability underflows adds nothing
                    if (kStats && p != 0.0f) part += p * (d - logf(ts.s) - ((zt[e] - all.m) * a.inv_t - ln_s));
                }
                if (kGrad && ahead[e].entry < a.K) {
                    sm.col[turn][ahead[e].entry] = used[e] ? col[e] : -1;
                    sm.p[turn][ahead[e].entry] = p;
                }
            }
            if (kStats) {
                part = warp_sum(part);
                if (l == 0) sm.red[turn][warp] = part;
            }
        }
        if (MODE == kDistillForward && tid == 0 && rank == 0 && a.lse != nullptr)
            a.lse[row] = all.s == 0.0f ? kNegInf : all.m * a.inv_t + ln_s;

        const float wt = w * a.t;
        if (kGrad) {
            // w t q = scale * 2^(z c - mc), or 2^((z - m) c) where the plain form was needed,
            // with scale = w t / s; from a kept normaliser scale * 2^((z - m) c) too, with m = lse t and
            // what its rounding leaves in scale, or as in the plain form where lse does not serve
            float scale = 0.0f;
            if (!kStats && some) {
                all.m = __fmul_rn(lse, a.t);
                scale = wt * expf(-fmaf(lse, a.t, -all.m) * a.inv_t);
                if (!(fabsf(lse) < kLseLimit && fabsf(all.m) <= FLT_MAX)) {
                    all = plain_slice_of<T, false, kThreads, 4>(z, sl, ze, c, sm.plain);
                    all = stat_cluster<false, true>(all, c, sm.cta_plain, rank, ncta);
                    scale = wt / all.s;
                }
            } else if (some) {
                scale = wt / all.s;
            }
            const float nmc = kStats ? -shift_of(all.m, c) : -all.m;
            const auto wtq = [&](float x) { return scale * ex2(!kStats || plain ? (x - all.m) * c : fmaf(x, c, nmc)); };
            // (S itself for the teacher's columns, where q meets p: 2^rest taken off)
            const float sum_t = kStats && teacher && !plain ? all.s * expf(-shift_rest(all.m, c) * kLn2) : all.s;
            const bool vec_out = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15u) == 0;
            const uint64_t mul2 = pack_f32x2(c, c), add2 = pack_f32x2(nmc, nmc), scale2 = pack_f32x2(scale, scale);
            T* out = dz + sl.head + (static_cast<size_t>(sl.v0) + tid) * kVec;
            for (int b = 0; b < batches; ++b, out += kUnroll * kThreads * kVec) {
                cp_async_wait<kDepth - 1>();
                uint4 v[kUnroll];
                stream.read(slot, sl, b, v);
                stream.fetch();
                slot = St::next(slot);
                const int n = sl.v1 - sl.v0 - b * (kUnroll * kThreads) - tid;   // vectors left from this one on
                if (some && !plain) {
#pragma unroll
                    for (int u = 0; u < kUnroll; ++u) {
                        float x[kVec];
                        Elem<T>::unpack(v[u], x);
#pragma unroll
                        for (int j = 0; j < kVec; j += 2) {
                            const uint64_t z2 = pack_f32x2(x[j], x[j + 1]);
                            const uint64_t y = kStats ? fma_f32x2(z2, mul2, add2) : mul_f32x2(add_f32x2(z2, add2), mul2);
                            float y0, y1;
                            unpack_f32x2(y, y0, y1);
                            unpack_f32x2(mul_f32x2(pack_f32x2(ex2(y0), ex2(y1)), scale2), x[j], x[j + 1]);
                        }
                        if (u * kThreads < n) store_vec<T>(out + u * (kThreads * kVec), Elem<T>::pack(x), vec_out);
                    }
                } else {   // a row out of use, or summed in the plain form
#pragma unroll 1
                    for (int u = 0; u * kThreads < n && u < kUnroll; ++u) {
                        const uint4 w = u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3];
                        float x[kVec];
                        Elem<T>::unpack(w, x);
#pragma unroll
                        for (int j = 0; j < kVec; ++j) x[j] = some ? wtq(x[j]) : 0.0f;
                        store_vec<T>(out + u * (kThreads * kVec), Elem<T>::pack(x), vec_out);
                    }
                }
            }
            if (edge >= 0) dz[edge] = Elem<T>::store(some ? wtq(ze) : 0.0f);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                end.col[e] = used[e] && col[e] >= sl.lo && col[e] < sl.hi ? col[e] : -1;
                end.base[e] = kStats ? wt * expf((zt[e] - all.m) * a.inv_t) / sum_t : wtq(zt[e]);
            }
            end.wt = wt;
            end.dz = dz;
        }
        end.loss_w = some ? wt * a.t : 0.0f;
        end.row = row;
    }
    __syncthreads();
    finish(turn ^ 1);
}

template <class T, DistillMode MODE>
static cudaError_t launch(const DistillArgs& a, cudaStream_t s) {
    using St = Stream<T, kThreads, kUnroll, kDepth>;
    const long long bytes = static_cast<long long>(a.C) * sizeof(T);
    // (the loss alone is split as the loss with its gradient, so that both give the same sums)
    const RowCost cost = {16 << 10, 16 << 10, MODE != kDistillBackward};
    if (a.K <= kThreads) return launch_rows<DistillArgs, distill_kernel<T, MODE, 1>>(a, bytes, cost, kThreads, St::kBytes, s);
    return launch_rows<DistillArgs, distill_kernel<T, MODE, 2>>(a, bytes, cost, kThreads, St::kBytes, s);
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
    set_floor(type, a.inv_t * kLog2e, a.floor, a.floor2);
    switch (type) {
        case DH_T_BF16: return launch_mode<__nv_bfloat16>(a, mode, s);
        case DH_T_F16: return launch_mode<__half>(a, mode, s);
        default: return launch_mode<float>(a, mode, s);
    }
}

}  // namespace dh
