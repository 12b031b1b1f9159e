// Token log-probabilities of logits rows: log p of given tokens, the entropy,
// the normaliser and the top alternatives, from one pass over the logits.
//
//   d = (z - max z) / t,  S = sum e^d,
//   lse = max z / t + ln S,  H = ln S - (sum e^d d) / S,  log p(j) = d_j - ln S.
//
// Persistent clusters of 1..8 CTAs take the rows in turn. Every thread streams
// its vectors through shared memory and keeps their running statistics
// (dh_rows.cuh), joined by shuffles, through shared memory and, between CTAs,
// by stores into the peers' shared memory. The row is read once.
//
// Top alternatives. The largest logit of each thread's vectors comes out of
// the statistics. A value T that at least k of a CTA's 256 thread maxima reach
// is a lower bound on the CTA's k-th largest logit, so only the vectors of the
// threads whose maximum reaches T can hold one of its top k. T is found bit by
// bit stopping at a count of up to k + k/8 + 2; those
// threads' vectors (about k/256 of the slice, still in L2) are read again by the
// whole CTA, elements >= T become candidates, and the rank of each among
// the candidates is counted. Candidates are 64-bit keys (ordered value, then
// the complement of the column), so equal logits go to the lowest column and
// the arrival order does not matter. More than kCand candidates (rows of many
// equal values) or a NaN send the CTA to an exact radix selection over its slice
// instead. The CTAs' sorted lists are merged by the first CTA.
//
// Bound: latency, with three CTAs per SM to hide it: 4,096 rows of 64,026 bf16, 20
// alternatives, take 130 us, 4.0 of the measured 6.8 TB/s (77 us). The SMs issue in 56
// of 100 cycles and DRAM is busy in 42; the largest stall is the barriers of a row's
// ends. 7 instructions per 32 logits go into the statistics, about 1.5 into reading the
// candidates' vectors again and 5,600 into a row's ends. Three CTAs of 256 threads per SM, so that
// one row's ends run under the others' streaming (two CTAs of 512 threads: 169 us,
// 256 threads twice 159, four times 149, 128 threads four times 183), with two batches of
// four vectors in flight each (two vectors, four batches: 150; four and three: 169).
// Steps: one kernel per row without a stream 164 us; logits streamed, exponents by
// one multiply-add and sums in pairs 140; the k-th bound searched in one warp and
// down to k + k/8 + 2 131. One row of 64,026 f32: 9.7 us, on 8 CTAs.
#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_rows.cuh"

namespace dh {
namespace rows {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCand = 1024;   // candidates a CTA ranks by counting
constexpr int kFew = 256;     // columns that are all candidates (4 x 1,000 f32, k = 20: 11.7 us with 1,024 here, 10.1 with 256)
constexpr int kUnroll = 4;    // vectors per batch and thread
constexpr int kDepth = 2;     // batches in flight: 32 KB per CTA
constexpr int kPerSm = 3;     // CTAs per SM

struct LogprobSmem {
    float warp[2][kWarps][3];
    float plain[kWarps][3];
    float cta[2][kMaxCluster][3];
    float cta_plain[kMaxCluster][3];
    uint32_t key[kThreads];   // the threads' maxima
    uint32_t bound;
    int n_active, n_cand, n_top;
    uint32_t sel_bin, sel_need;
    int scan[kWarps];
    int active[kThreads];
    uint32_t hist[256];
    alignas(16) unsigned long long cand[kCand];
    unsigned long long top[DH_MAX_TOP];                     // this CTA's list, descending; 0 = none
    unsigned long long peers[2][kMaxCluster][DH_MAX_TOP];   // the first CTA: every CTA's list
};

__device__ __forceinline__ void push_candidate(LogprobSmem& sm, float z, uint32_t col) {
    const int at = atomicAdd(&sm.n_cand, 1);
    if (at < kCand) sm.cand[at] = argmax_key(ordered_key(z), col);
}

// Sort the n <= kCand candidates (distinct keys) and keep the k largest.
__device__ __forceinline__ void rank_candidates(LogprobSmem& sm, int n, int k) {
    for (int e = threadIdx.x; e < k; e += kThreads) sm.top[e] = 0ull;
    if (threadIdx.x == 0) {
        sm.n_top = min(n, k);
        if ((n & 1) && n < kCand) sm.cand[n] = 0ull;   // read in pairs
    }
    __syncthreads();
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(sm.cand);
    for (int e = threadIdx.x; e < n; e += kThreads) {
        const unsigned long long mine = sm.cand[e];
        int above = 0;
#pragma unroll 4
        for (int j = 0; j < (n + 1) / 2; ++j) {
            const ulonglong2 p = pairs[j];
            above += (p.x > mine) + (p.y > mine);
        }
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

// A bound that at least k of the CTA's keys (a maximum per thread) reach, and that at
// most k + k/8 + 2 reach where the keys allow it; 0 where fewer than k lie above
// -inf. The first warp looks for it bit by bit, from the bits that all keys above
// -inf share: a count of 256 keys in one warp's registers is a few
// instructions, where a barrier per bit is tens of cycles (4,096 x 64,026: 143 -> 137 us).
__device__ __forceinline__ uint32_t kth_bound(LogprobSmem& sm, uint32_t key, int k) {
    const uint32_t floor_key = ordered_key(kNegInf);
    sm.key[threadIdx.x] = key;
    __syncthreads();
    if (threadIdx.x < 32) {
        constexpr int kPer = kThreads / 32;
        uint32_t mine[kPer], lo = 0xFFFFFFFFu, hi = 0u;
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            mine[i] = sm.key[threadIdx.x + 32 * i];
            const bool in = mine[i] > floor_key;
            lo = in ? min(lo, mine[i]) : lo;
            hi = in ? max(hi, mine[i]) : hi;
            n += in;
        }
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        uint32_t t = 0;
        if (n >= k) {
            lo = __reduce_min_sync(0xFFFFFFFFu, lo);
            hi = __reduce_max_sync(0xFFFFFFFFu, hi);
            int bit = 31 - __clz(static_cast<int>(lo ^ hi));
            t = bit >= 31 ? 0u : lo >> (bit + 1) << (bit + 1);
#pragma unroll 1
            for (; bit >= 0 && n > k + k / 8 + 2; --bit) {
                const uint32_t up = t | (1u << bit);
                int c = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) c += mine[i] >= up;
                c = __reduce_add_sync(0xFFFFFFFFu, c);
                if (c >= k) {
                    t = up;
                    n = c;
                }
            }
        }
        if (threadIdx.x == 0) sm.bound = t;
    }
    __syncthreads();
    return sm.bound;
}

// The CTA's k largest logits into sm.top. `mx` is this thread's largest logit and `ze`
// its edge logit (-inf: none).
template <class T>
__device__ __forceinline__ void cta_top(LogprobSmem& sm, const T* z, const Slice& sl, int edge, float ze, float mx, bool nan,
                                        int k) {
    constexpr int kVec = Elem<T>::kVec;
    if (nan) {
        radix_top(sm, z, sl.lo, sl.hi, k);
        return;
    }
    const uint32_t key = ordered_key(mx);
    uint32_t bound_key = 0;
    if (threadIdx.x == 0) sm.n_active = sm.n_cand = 0;
    if (sl.hi - sl.lo > kFew) {
        bound_key = kth_bound(sm, key, k);
    }
    __syncthreads();
    // the threads that reach the bound, each warp's in a row
    const bool active = key >= bound_key && key > ordered_key(kNegInf) && sl.v0 + static_cast<int>(threadIdx.x) < sl.v1;
    const unsigned votes = __ballot_sync(0xFFFFFFFFu, active);
    int at = 0;
    if ((threadIdx.x & 31) == 0 && votes != 0u) at = atomicAdd(&sm.n_active, __popc(votes));
    at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(votes & ((1u << (threadIdx.x & 31)) - 1u));
    if (active) sm.active[at] = threadIdx.x;
    if (edge >= 0 && ze > kNegInf && ordered_key(ze) >= bound_key) push_candidate(sm, ze, static_cast<uint32_t>(edge));
    __syncthreads();
    // their vectors (i of thread a: v0 + a + i * kThreads) over the whole CTA, four at a time;
    // the bound as a value (below every logit's key: any logit above -inf)
    const float bound = bound_key <= ordered_key(kNegInf) ? -FLT_MAX : ordered_value(bound_key);
    const int per = (sl.v1 - sl.v0 + kThreads - 1) / kThreads, total = sm.n_active * per;
#pragma unroll 1
    for (int f0 = threadIdx.x; f0 < total; f0 += 4 * kThreads) {
        uint4 w[4][1];
        int v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = f0 + i * kThreads, a = f / per;
            v[i] = f < total ? sl.v0 + sm.active[a] + (f - a * per) * kThreads : sl.v1;
            w[i][0] = v[i] < sl.v1 ? ld_stream_v4(z + sl.head + static_cast<size_t>(v[i]) * kVec) : neg_inf_vec<T>();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (Elem<T>::template max_of<1>(w[i]) < bound) continue;
            float x[kVec];
            Elem<T>::unpack(w[i][0], x);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (x[j] >= bound) push_candidate(sm, x[j], static_cast<uint32_t>(sl.head + v[i] * kVec + j));
        }
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

// How many keys of a descending list lie above `key`.
__device__ __forceinline__ int list_count(const unsigned long long* list, int k, unsigned long long key) {
    int lo = 0, hi = k;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] > key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <class T>
__global__ void __launch_bounds__(kThreads, kPerSm) token_logprobs_kernel(const LogprobArgs a) {
    using St = Stream<T, kThreads, kUnroll, kDepth>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ LogprobSmem sm;
    const unsigned lg = a.lg, ncta = 1u << lg, rank = ncta > 1 ? cluster_ctarank() : 0u;
    const int first = blockIdx.x >> lg, stride = gridDim.x >> lg;
    const float c = a.inv_t * kLog2e;
    St stream;
    stream.start(static_cast<const T*>(a.z), a.ld, a.M, a.C, rank, lg, first, stride, ring);
    IdAhead tokens = {a.tokens, a.row_of, a.G, a.V, a.C, a.M, stride, static_cast<int>(threadIdx.x), -1, -1, -1};
    if (rank == 0) tokens.start(first);
    if (ncta > 1) {   // every peer runs before its shared memory is written
        cluster_arrive_release();
        cluster_wait_acquire();
    }
    uint32_t slot = 0;
    int turn = 0;
    const T* z = static_cast<const T*>(a.z) + static_cast<size_t>(first) * a.ld;
    Slice sl = make_slice(z, a.C, rank, lg);
    for (int row = first; row < a.M; row += stride, turn ^= 1, z += static_cast<size_t>(stride) * a.ld) {
        if (!stream.alike) sl = make_slice(z, a.C, rank, lg);
        const int edge = edge_column(sl, a.C, rank, ncta);
        float zt = kNegInf, ze = kNegInf;
        int col = -1;
        if (rank == 0) col = tokens.take(row);
        if (col >= 0) zt = Elem<T>::load(z + col);
        if (edge >= 0) ze = Elem<T>::load(z + edge);

        Stat st = {a.floor, 0.0f, 0.0f};
        float top = ze;
        const int batches = St::batches_of(sl);
        for (int b = 0; b < batches; ++b) {
            cp_async_wait<kDepth - 1>();
            uint4 w[kUnroll];
            stream.read(slot, sl, b, w);
            stream.fetch();
            slot = St::next(slot);
            stat_add<T, true, kUnroll>(st, top, w, c, a.floor2);
        }
        if (edge >= 0) stat_add1<true>(st, ze, c, a.floor);

        stat_leave(stat_warp<true, false>(st, c), sm.warp[turn]);
        __syncthreads();
        const Stat mine = stat_gather<true, false>(kWarps, c, sm.warp[turn], a.floor);
        Stat all = stat_cluster<true, false>(mine, c, sm.cta[turn], rank, ncta);
        float rest = 0.0f;   // m c less its rounding, which the sums carry
        if (stat_fits(all.m, c, a.floor)) {
            rest = shift_rest(all.m, c);
        } else {
            // masked throughout (and no NaN), or summed in the plain form
            if (row_top<kThreads>(top, sm.plain, sm.cta_plain, rank, ncta) == kNegInf && all.s == all.s) {
                all = Stat{0.0f, 0.0f, 0.0f};
            } else {
                all = plain_slice<T, true, kThreads>(z, sl, ze, c, sm.plain);
                all = stat_cluster<true, true>(all, c, sm.cta_plain, rank, ncta);
            }
        }
        if (a.k > 0) {
            cta_top(sm, z, sl, edge, ze, top, mine.s != mine.s, a.k);
            if (ncta > 1) {
                for (int i = threadIdx.x; i < a.k; i += kThreads)
                    st_cluster_u64(cluster_map(&sm.peers[turn][rank][i], 0), sm.top[i]);
                cluster_arrive_release();
                cluster_wait_acquire();
            }
        }
        if (rank != 0) continue;

        // results (a warp without any only passes the barrier at the end)
        const bool empty = all.s == 0.0f;
        float ln_s = 0.0f;
        if (static_cast<int>(threadIdx.x & ~31u) < max(max(a.G, a.k * static_cast<int>(ncta)), 1)) ln_s = logf(all.s) - rest * kLn2;
        if (threadIdx.x == 0) {
            if (a.lse != nullptr) a.lse[row] = empty ? kNegInf : all.m * a.inv_t + ln_s;
            // the mean of (z - max) / t is (s1 / s - rest) ln 2
            if (a.entropy != nullptr) a.entropy[row] = empty ? 0.0f : ln_s - (all.s1 / all.s - rest) * kLn2;
        }
        for (int g = threadIdx.x; g < a.G; g += kThreads) {
            const size_t at = static_cast<size_t>(row) * a.G + g;
            if (g >= kThreads) {
                col = column_of(a.tokens[at], a.row_of, a.V, a.C);
                zt = col >= 0 ? Elem<T>::load(z + col) : 0.0f;
            }
            a.logp[at] = col < 0 || empty ? kNegInf : (zt - all.m) * a.inv_t - ln_s;
        }
        // merge: the place of a key is its place in its own list plus the keys above it in the others
        const unsigned long long(*peers)[DH_MAX_TOP] = sm.peers[turn];
        for (int i = threadIdx.x; i < a.k * static_cast<int>(ncta); i += kThreads) {
            const unsigned r = static_cast<unsigned>(i) / a.k;
            int place = i - static_cast<int>(r) * a.k;
            const unsigned long long key = ncta > 1 ? peers[r][place] : sm.top[place];
            if (ncta > 1 && key != 0ull) {
                for (unsigned o = 0; o < ncta; ++o)
                    if (o != r) place += list_count(peers[o], a.k, key);
            }
            if (key == 0ull || place >= a.k) continue;
            const size_t at = static_cast<size_t>(row) * a.k + place;
            const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(key);
            a.top_logp[at] = (ordered_value(static_cast<uint32_t>(key >> 32)) - all.m) * a.inv_t - ln_s;
            a.top_ids[at] = a.idx != nullptr ? __ldg(a.idx + id) : static_cast<int32_t>(id);
        }
        if (a.k > 0) {   // places that no key took
            int n = ncta > 1 ? 0 : sm.n_top;
            for (unsigned r = 0; n < a.k && ncta > 1 && r < ncta; ++r)
                n += peers[r][a.k - 1] != 0ull ? a.k : list_count(peers[r], a.k, 0ull);
            for (int i = n + threadIdx.x; i < a.k; i += kThreads) {
                a.top_logp[static_cast<size_t>(row) * a.k + i] = kNegInf;
                a.top_ids[static_cast<size_t>(row) * a.k + i] = -1;
            }
            if (ncta == 1) __syncthreads();   // sm.top is read before the next row writes it
        }
    }
}

template <class T>
static cudaError_t launch(const LogprobArgs& a, cudaStream_t s) {
    using St = Stream<T, kThreads, kUnroll, kDepth>;
    return launch_rows<LogprobArgs, token_logprobs_kernel<T>>(a, static_cast<long long>(a.C) * sizeof(T), RowCost{32 << 10, 48 << 10, false},
                                                             kThreads, St::kBytes, s);
}

}  // namespace rows

cudaError_t launch_token_logprobs(LogprobArgs a, int type, cudaStream_t s) {
    using namespace rows;
    set_floor(type, a.inv_t * kLog2e, a.floor, a.floor2);
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
