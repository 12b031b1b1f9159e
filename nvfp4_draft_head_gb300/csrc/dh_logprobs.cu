// Token log-probabilities of logits rows: log p of given tokens, the entropy,
// the normaliser and the top alternatives, from one pass over the logits.
//
//   d = (z - max z) / t,  S = sum e^d,
//   lse = max z / t + ln S,  H = ln S - (sum e^d d) / S,  log p(j) = d_j - ln S.
//
// One cluster of 1..16 CTAs per row. Every thread keeps the running statistics
// of its vectors (dh_rows.cuh), joined by shuffles, through shared memory and,
// between CTAs, by stores into the peers' shared memory. The row is read once.
//
// Top alternatives. The largest logit of each thread's vectors comes out of
// the statistics. A value T that at least k of a CTA's 512 thread maxima reach
// is a lower bound on the CTA's k-th largest logit, so only the vectors of the
// threads whose maximum reaches T can hold one of its top k. T is found bit by
// bit with block-wide counts, stopping at a count of up to k + k/2 + 4; those
// threads' vectors (about k/512 of the slice, still in L2) are read again by the
// whole CTA, elements >= T become candidates, and the rank of each among
// the candidates is counted. Candidates are 64-bit keys (ordered value, then
// the complement of the column), so equal logits go to the lowest column and
// the arrival order does not matter. More than kCand candidates (rows of many
// equal values) or a NaN send the CTA to an exact radix selection over its
// slice instead. The CTAs' sorted lists are merged by the first CTA.
//
// Bound: HBM (C elements read per row); see the launcher for the measurements.
#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_rows.cuh"

namespace dh {
namespace rows {

constexpr int kCand = 1024;   // candidates a CTA ranks by counting
constexpr int kUnroll = 4;    // vectors in flight per thread

struct LogprobSmem {
    float warp[kWarps][3];
    float cta[kMaxCluster][3];
    int n_active, n_cand;
    uint32_t sel_bin, sel_need;
    int scan[kWarps];
    int active[kThreads];
    uint32_t hist[256];
    unsigned long long cand[kCand];
    unsigned long long top[DH_MAX_TOP];                  // this CTA's list, descending; 0 = none
    unsigned long long peers[kMaxCluster][DH_MAX_TOP];   // the first CTA: every CTA's list
};

__device__ __forceinline__ void push_candidate(LogprobSmem& sm, float z, uint32_t col) {
    const int at = atomicAdd(&sm.n_cand, 1);
    if (at < kCand) sm.cand[at] = argmax_key(ordered_key(z), col);
}

// Sort the n <= kCand candidates (distinct keys) and keep the k largest.
__device__ __forceinline__ void rank_candidates(LogprobSmem& sm, int n, int k) {
    for (int e = threadIdx.x; e < k; e += kThreads) sm.top[e] = 0ull;
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += kThreads) {
        const unsigned long long mine = sm.cand[e];
        int above = 0;
        for (int j = 0; j < n; ++j) above += sm.cand[j] > mine;
        if (above < k) sm.top[above] = mine;
    }
    __syncthreads();
}

// Exact selection over the columns [lo, hi) by radix: four 8-bit passes find
// the value of the k-th largest logit above -inf, then everything above it and
// the lowest columns among its equals are collected. Used for rows of many
// equal values and rows with NaN.
template <class T>
__device__ __noinline__ void radix_top(LogprobSmem& sm, const T* z, int lo, int hi, int k) {
    const uint32_t floor_key = ordered_key(kNegInf);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t prefix = 0;
    int need = k;      // how many of the elements under the prefix are wanted
    bool fewer = false;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) sm.hist[i] = 0;
        __syncthreads();
        for (int base = lo; base < hi; base += kThreads) {
            const int e = base + tid;
            const uint32_t key = e < hi ? ordered_key(Elem<T>::load(z + e)) : 0u;
            const bool in = e < hi && key > floor_key && (shift == 24 || (key >> (shift + 8)) == prefix);
            const uint32_t bin = in ? (key >> shift) & 0xFFu : 256u;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, bin);   // one add per warp and value
            if (in && lane == __ffs(same) - 1) atomicAdd(&sm.hist[bin], static_cast<uint32_t>(__popc(same)));
        }
        __syncthreads();
        if (tid == 0) {
            int left = need, b = 255;
            for (; b >= 0; --b) {
                const int n = static_cast<int>(sm.hist[b]);
                if (n >= left) break;
                left -= n;
            }
            sm.sel_bin = static_cast<uint32_t>(b);   // -1: fewer than k values above -inf (first pass only)
            sm.sel_need = static_cast<uint32_t>(left);
        }
        __syncthreads();
        const int b = static_cast<int>(sm.sel_bin);
        need = static_cast<int>(sm.sel_need);
        if (b < 0) {
            fewer = true;
            break;
        }
        prefix = shift == 24 ? static_cast<uint32_t>(b) : (prefix << 8) | static_cast<uint32_t>(b);
        __syncthreads();
    }
    // everything above the k-th value (or, where there are fewer than k, everything above -inf)
    const uint32_t kth = fewer ? floor_key : prefix;
    if (tid == 0) sm.n_cand = 0;
    __syncthreads();
    for (int e = lo + tid; e < hi; e += kThreads) {
        const float v = Elem<T>::load(z + e);
        if (ordered_key(v) > kth) push_candidate(sm, v, static_cast<uint32_t>(e));
    }
    __syncthreads();
    if (!fewer) {
        // the `need` lowest columns whose value is the k-th
        const int above = sm.n_cand;
        int found = 0;
        for (int base = lo; base < hi && found < need; base += kThreads) {
            const int e = base + tid;
            const float v = e < hi ? Elem<T>::load(z + e) : 0.0f;
            const bool eq = e < hi && ordered_key(v) == kth;
            const unsigned votes = __ballot_sync(0xFFFFFFFFu, eq);
            if (lane == 0) sm.scan[warp] = __popc(votes);
            __syncthreads();
            int before = found, total = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before += sm.scan[w];
                total += sm.scan[w];
            }
            const int at = before + __popc(votes & ((1u << lane) - 1u));
            if (eq && at < need) sm.cand[above + at] = argmax_key(kth, static_cast<uint32_t>(e));
            found += total;
            __syncthreads();
        }
        if (tid == 0) sm.n_cand = above + need;
        __syncthreads();
    }
    rank_candidates(sm, sm.n_cand, k);
}

// The CTA's k largest logits into sm.top. `mx` is this thread's largest logit.
template <class T>
__device__ __forceinline__ void cta_top(LogprobSmem& sm, const T* z, const Slice& sl, int edge, float mx, bool nan, int k) {
    constexpr int kVec = Elem<T>::kVec;
    if (nan) {
        radix_top(sm, z, sl.lo, sl.hi, k);
        return;
    }
    const uint32_t key = ordered_key(mx);
    uint32_t T_key = 0;
    if (threadIdx.x == 0) sm.n_active = sm.n_cand = 0;
    if (sl.hi - sl.lo > kCand) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t t = T_key | (1u << bit);
            const int n = __syncthreads_count(key >= t);
            if (n >= k) {
                T_key = t;
                if (n <= k + k / 2 + 4) break;
            }
        }
    }
    __syncthreads();
    if (key >= T_key && sl.v0 + static_cast<int>(threadIdx.x) < sl.v1)
        sm.active[atomicAdd(&sm.n_active, 1)] = threadIdx.x;
    if (edge >= 0) {
        const float v = Elem<T>::load(z + edge);
        if (v > kNegInf && ordered_key(v) >= T_key) push_candidate(sm, v, static_cast<uint32_t>(edge));
    }
    __syncthreads();
    // vector i of active thread a is v0 + a + i * kThreads
    const int per = (sl.v1 - sl.v0 + kThreads - 1) / kThreads, total = sm.n_active * per;
    for (int f = threadIdx.x; f < total; f += kThreads) {
        const int a = f / per, v = sl.v0 + sm.active[a] + (f - a * per) * kThreads;
        if (v >= sl.v1) continue;
        const int col = sl.head + v * kVec;
        float x[kVec];
        Elem<T>::unpack(ld_stream_v4(z + col), x);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (x[j] > kNegInf && ordered_key(x[j]) >= T_key) push_candidate(sm, x[j], static_cast<uint32_t>(col + j));
    }
    __syncthreads();
    const int n = sm.n_cand;
    if (n > kCand) {
        __syncthreads();
        radix_top(sm, z, sl.lo, sl.hi, k);
    } else {
        rank_candidates(sm, n, k);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const LogprobArgs a) {
    constexpr int kVec = Elem<T>::kVec;
    __shared__ LogprobSmem sm;
    const unsigned rank = cluster_ctarank(), ncta = a.ncta;
    const int row = blockIdx.x / ncta;
    if (ncta > 1) cluster_arrive_release();
    const T* z = static_cast<const T*>(a.z) + static_cast<size_t>(row) * a.ld;
    const Slice sl = make_slice(z, a.C, rank, ncta);
    const float c = a.inv_t * kLog2e;

    Stat st = stat_empty();
    for (int v0 = sl.v0 + threadIdx.x; v0 < sl.v1; v0 += kUnroll * kThreads) {
        uint4 w[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * kThreads;
            w[u] = v < sl.v1 ? ld_stream_v4(z + sl.head + static_cast<size_t>(v) * kVec) : neg_inf_vec<T>();
        }
        float x[kUnroll * kVec];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) Elem<T>::unpack(w[u], reinterpret_cast<float(&)[kVec]>(x[u * kVec]));
        stat_add<true>(st, x, c);
    }
    const int edge = edge_column(sl, a.C, rank, ncta);
    if (edge >= 0) stat_add1<true>(st, Elem<T>::load(z + edge), c);

    const Stat mine = stat_block<true>(st, c, sm.warp);
    if (a.k > 0) {
        // a NaN in the slice (its values alone decide: an infinity makes s a NaN too, and is selected exactly)
        cta_top(sm, z, sl, edge, st.m, mine.s != mine.s, a.k);
    }
    const Stat all = stat_cluster<true>(mine, c, sm.cta, rank, ncta);
    if (a.k > 0 && ncta > 1) {
        for (int i = threadIdx.x; i < a.k; i += kThreads)
            st_cluster_u64(cluster_map(&sm.peers[rank][i], 0), sm.top[i]);
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    if (rank != 0) return;

    // ln S with S = sum e^((z - max)/t)
    const bool empty = all.s == 0.0f;
    const float ln_s = logf(all.s);
    if (threadIdx.x == 0) {
        if (a.lse != nullptr) a.lse[row] = empty ? kNegInf : all.m * a.inv_t + ln_s;
        if (a.entropy != nullptr) a.entropy[row] = empty ? 0.0f : ln_s - all.s1 * kLn2 / all.s;
    }
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        const size_t at = static_cast<size_t>(row) * a.G + g;
        const int col = column_of(a.tokens[at], a.row_of, a.V, a.C);
        a.logp[at] = col < 0 || empty ? kNegInf : (Elem<T>::load(z + col) - all.m) * a.inv_t - ln_s;
    }
    // merge: the place of a key is its place in its own list plus the keys above it in the others
    for (int i = threadIdx.x; i < a.k * static_cast<int>(ncta); i += kThreads) {
        const unsigned r = static_cast<unsigned>(i) / a.k;
        int place = i - static_cast<int>(r) * a.k;
        const unsigned long long key = ncta > 1 ? sm.peers[r][place] : sm.top[place];
        if (ncta > 1 && key != 0ull) {
            for (unsigned o = 0; o < ncta; ++o) {
                if (o == r) continue;
                int lo = 0, hi = a.k;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (sm.peers[o][mid] > key) lo = mid + 1;
                    else hi = mid;
                }
                place += lo;
            }
        }
        if (key == 0ull || place >= a.k) continue;
        const size_t at = static_cast<size_t>(row) * a.k + place;
        const uint32_t col = 0xFFFFFFFFu - static_cast<uint32_t>(key);
        a.top_logp[at] = (ordered_value(static_cast<uint32_t>(key >> 32)) - all.m) * a.inv_t - ln_s;
        a.top_ids[at] = a.idx != nullptr ? __ldg(a.idx + col) : static_cast<int32_t>(col);
    }
    // places that no key took
    int n = 0;
    if (a.k > 0) {
        for (unsigned r = 0; r < ncta; ++r) {
            int lo = 0, hi = a.k;
            const unsigned long long* list = ncta > 1 ? sm.peers[r] : sm.top;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] != 0ull) lo = mid + 1;
                else hi = mid;
            }
            n += lo;
        }
        for (int i = n + threadIdx.x; i < a.k; i += kThreads) {
            a.top_logp[static_cast<size_t>(row) * a.k + i] = kNegInf;
            a.top_ids[static_cast<size_t>(row) * a.k + i] = -1;
        }
    }
}

// CTAs per row: enough to give the GPU two CTAs per SM, each with at least
// 8 KB of the row to read (below that a slice's fixed costs outweigh it).
int cluster_size(int M, long long row_bytes) {
    const int sms = sm_count();
    int n = 1;
    while (n < 8 && static_cast<long long>(M) * n * 2 <= 2ll * sms && row_bytes / (2 * n) >= 8192) n *= 2;
    return n;
}

template <class T>
static cudaError_t launch(const LogprobArgs& a, cudaStream_t s) {
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
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a);
}

}  // namespace rows

cudaError_t launch_token_logprobs(LogprobArgs a, int type, cudaStream_t s) {
    using namespace rows;
    a.ncta = static_cast<unsigned>(cluster_size(a.M, static_cast<long long>(a.C) * (type == DH_T_F32 ? 4 : 2)));
    switch (type) {
        case DH_T_BF16: return launch<__nv_bfloat16>(a, s);
        case DH_T_F16: return launch<__half>(a, s);
        default: return launch<float>(a, s);
    }
}

__global__ void row_map_kernel(const int32_t* __restrict__ idx, int n, int32_t* __restrict__ row_of, int V) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int id = idx[i];
    if (id >= 0 && id < V) row_of[id] = i;
}

cudaError_t launch_row_map(const int32_t* idx, int n, int32_t* row_of, int V, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(row_of, 0xFF, static_cast<size_t>(V) * sizeof(int32_t), s);
    if (e != cudaSuccess) return e;
    row_map_kernel<<<(n + 255) / 256, 256, 0, s>>>(idx, n, row_of, V);
    return cudaGetLastError();
}

}  // namespace dh
