// The tensor-core product under the operators of many tokens with 16-bit and FP8 operands
// (cross entropy, FP8 blocks): a persistent kernel whose operands come row-major from global
// memory by tensor maps (TMA, 128-byte swizzle) and whose results each operator takes from
// tensor memory in its own way (Op::tile).
//
// A tile is 128 P rows x TN columns, P the CTAs that share it. With a pair (P = 2) each CTA
// loads its 128 rows of A and half of B: two thirds of the bytes that two single CTAs need
// for the same 256 x TN, at 32 bytes of K per instruction. Single CTAs are for
// products with an accumulator per step of K, which would wait for a pair's hand-over between
// its CTAs. A stage is 128 bytes of K (64 16-bit elements, 128 FP8). An operand is K-major (its
// rows run along the contraction) or MN-major (its rows run along M or N, one row per step of the
// contraction): both gradients of a layer then read the matrices as they lie, without transposed
// copies.
//
// Warps: eight or sixteen epilogue warps (four groups of 32 lanes, parts of the columns), a
// producer's, one or two issuers' (a pair: rank 0's alone work). Every wait is bounded; who gives
// up sets the CTA's abort flag and the caller's error word, and the others follow.
//
// What it reaches: 16-bit operands in pairs keep the tensor pipe busy for 95 to 97 of 100 cycles
// (1,024 x 64,064 x 2,560); FP8 in single CTAs, 256 wide, with a sum of its own for every 128
// features, 56 (2,048 x 64,064 x 2,560 270 us): a step lands 48 KB in an SM's shared
// memory while its instructions take 512 cycles, and hands over an accumulator of half the tensor
// memory. What changes that balance was measured there
// (8,192 x 64,064): pairs 1,380 us, whose hand-over crosses CTAs; halves of the columns with
// accumulators of their own 1,176, which read A twice; single CTAs 1,150.
#pragma once

#include <atomic>
#include <utility>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_tcgen05.cuh"

namespace dh {
namespace gemm {

constexpr int kRows = 128;            // rows of a CTA's part of a tile: the lanes of tensor memory
constexpr int kStageBytes = 128;      // bytes of K in a stage
constexpr int kWaitSlices = 64;
constexpr uint32_t kDrainRounds = kWaitLimit / kWaitSlices;

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// What a launch multiplies: tiles, the steps of K, and where the operands start in their maps.
// The first `whole` tiles are multiplied whole; each of the rest in `splits` parts of
// split_steps steps of K (the last may have fewer), so that the last round of tiles over the SMs
// can be a full one.
struct Shape {
    int tiles_m, tiles_n, whole, splits;
    int steps, split_steps;
    int a_mn, a_k, b_mn, b_k;       // first row (M / N) and first element of K of each operand
    unsigned int* error;            // DH_DEVERR_* word or null
    uint32_t rounds;                // self-test: tries of a bounded wait, times kWaitSlices (0: a product's own)
    int idle;                       // self-test: the role that does nothing (-1: none)
    int chunk;                      // steps of K that share an accumulator, where the operator leaves it to the launch
    __host__ __device__ int tiles() const { return tiles_m * tiles_n; }
    __host__ __device__ int units() const { return whole + (tiles() - whole) * splits; }
};

constexpr int kPerLaunch = 0;   // of an operator's kChunk

enum Role { kRoleProducer, kRoleIssuer, kRoleEpilogue };

// Tiles that are in work at the same time share operands in L2: groups of kGroup rows of
// tiles, columns along a group.
constexpr int kGroup = 8;
struct Tile { int m, n, split, k0, steps; };   // split: the part, -1 for a whole tile; k0: its first step
__device__ __forceinline__ Tile tile_at(const Shape& s, int i) {
    Tile t = {0, 0, -1, 0, s.steps};
    if (i >= s.whole) {
        const int rest = s.tiles() - s.whole, j = i - s.whole;
        t.split = j / rest;
        t.k0 = t.split * s.split_steps;
        t.steps = min(s.split_steps, s.steps - t.k0);
        i = s.whole + j - t.split * rest;
    }
    const int g = i / (kGroup * s.tiles_n), rows = min(kGroup, s.tiles_m - g * kGroup);
    i -= g * kGroup * s.tiles_n;
    t.n = i / rows;
    t.m = g * kGroup + i - t.n * rows;
    return t;
}
// The place of tile (m, n) in that order.
__host__ __device__ inline int tile_index(int tiles_m, int tiles_n, int m, int n) {
    const int g = m / kGroup, rows = tiles_m - g * kGroup < kGroup ? tiles_m - g * kGroup : kGroup;
    return g * kGroup * tiles_n + n * rows + m - g * kGroup;
}

template <int P, int TN, int ELEM, bool A_MN, bool B_MN, int EPI = 8, int ISSUERS = 1>
struct Layout {
    static constexpr int kP = P, kTN = TN, kElem = ELEM;
    static constexpr int kEpiWarps = EPI, kProducer = EPI, kIssuer = EPI + 1, kIssuers = ISSUERS, kThreads = 32 * (EPI + 1 + ISSUERS);
    static constexpr int kPart = TN / (EPI / 4);                        // columns of an epilogue warp
    static constexpr bool kAMn = A_MN, kBMn = B_MN;
    static constexpr int kK = kStageBytes / ELEM;                       // elements of K per stage
    static constexpr int kSpan = 128 / ELEM;                            // elements of an MN-major box's rows
    static constexpr int kBRows = TN / P;                               // columns of B that a CTA holds
    static constexpr int kABytes = kRows * kStageBytes, kBBytes = kBRows * kStageBytes;
    static constexpr int kBytes = kABytes + kBBytes;
    // stages: a multiple of the issuers, which take the steps in turn (a wait by parity needs a
    // waiter that has seen the slot's phase before)
    static constexpr int kFit = (227 * 1024 - 1024 - 1024) / kBytes, kStages = (kFit < 8 ? kFit : 8) / ISSUERS * ISSUERS;
    static constexpr int kSmem = kStages * kBytes + 1024;
    static constexpr int kBuffers = 512 / TN < 4 ? 512 / TN : 4;        // accumulators in tensor memory
    static_assert(!(A_MN && kRows % kSpan != 0) && !(B_MN && kBRows % kSpan != 0), "whole boxes");
    static_assert(kStages <= 8 && kBytes % 1024 == 0 && TN % 32 == 0 && kStages >= 3, "stage layout");
    static_assert(kBuffers % ISSUERS == 0, "and the accumulators");
};

struct Sync {
    uint64_t full[8], empty[8], acc_full[4], acc_empty[4], issued;
    uint32_t tmem;
    unsigned int abort;
    uint32_t copies;   // self-test: stages that the producer filled
};

// One lane of a converged warp, known to the compiler as such: what it issues takes its
// operands from uniform registers. (Loops of one lane alone, with the same instructions, took
// 870 cycles for an issuer's step.)
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0u;
}

// A bounded wait that gives up at once when another role of this CTA has.
static __device__ __noinline__ bool wait_longer(volatile unsigned int* abort, uint64_t* bar, uint32_t parity, uint32_t rounds,
                                                unsigned int* error) {
    for (int i = 0; i < kWaitSlices; ++i) {
        if (mbar_wait(bar, parity, rounds)) return true;   // (about 1 us a round)
        if (*abort != 0u) return false;
    }
    *abort = 1u;
    if (error != nullptr) atomicOr(error, kDevErrTimeout);
    return false;
}
__device__ __forceinline__ bool wait_or_abort(Sync& sy, uint64_t* bar, uint32_t parity, const Shape& s) {
    return mbar_wait<false>(bar, parity, 1) || wait_longer(&sy.abort, bar, parity, s.rounds, s.error);
}

// A box of a tensor map into this CTA's shared memory, completing on `bar` (with a pair: a
// shared::cluster address, rank 0's barrier).
template <int P>
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
    if constexpr (P == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
                     " [%0], [%1, {%2, %3}], [%4], %5;"
                     :: "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
                     " [%0], [%1, {%2, %3}], [%4], %5;"
                     :: "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}

__device__ __forceinline__ uint64_t policy_evict_last() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Arrive on rank 0's barrier, with the default scope, this CTA's. What the arrival has to order are
// tensor-memory loads alone: those have returned (tmem_load_wait) before the warps arrive that this
// thread has waited for, and the tcgen05 fences on both sides keep them there. Released at cluster scope
// it would wait for this thread's global accesses in flight too, and a step of the FP8 product took
// 1.05 us.
__device__ __forceinline__ void arrive_rank0(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_map(bar, 0)) : "memory");
}

// An operand's part of a stage: `rows` of M or N from `mn`, kK elements of K from `k`.
template <class L, bool MN>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, int rows, int mn, int k, uint32_t bar,
                                             uint64_t policy) {
    if constexpr (!MN) {
        tma_2d<L::kP>(dst, map, k, mn, bar, policy);
    } else {
        for (int i = 0; i < rows / L::kSpan; ++i)   // boxes of kSpan elements x kK rows
            tma_2d<L::kP>(dst + i * L::kK * 128, map, mn + i * L::kSpan, k, bar, policy);
    }
}

// The epilogue warps' turn through the accumulators.
// (L: any of a launch's layouts, which differ in their operands alone)
template <class L>
struct Acc {
    Sync& sy;
    const Shape& shape;
    uint32_t tmem, n = 0;
    __device__ Acc(Sync& s, const Shape& sh, uint32_t t) : sy(s), shape(sh), tmem(t) {}
    // Waits for the next accumulator: its first column, or ~0 if the wait gave up.
    __device__ __forceinline__ uint32_t next() {
        const uint32_t b = n % L::kBuffers;
        const bool ok = wait_or_abort(sy, &sy.acc_full[b], (n / L::kBuffers) & 1, shape);
        if (!__all_sync(0xFFFFFFFFu, ok)) return ~0u;
        tc::fence_after_sync();
        return tmem + b * L::kTN;
    }
    // This warp has read the accumulator (all of its loads waited for).
    __device__ __forceinline__ void release() {
        tc::fence_before_sync();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sy.acc_empty[n % L::kBuffers]);
        ++n;
    }
};

// Op: Layout, Args (with `Shape shape`), kFormat (idesc_f), kChunk (steps of K that share an
// accumulator: results that are scaled step by step take 1; kPerLaunch: Shape's chunk, a power of
// two), kAKeep / kBKeep (the operand is read by other tiles too: kept in L2), and tile(args, tile,
// warp, lane, rank, acc), false when a wait gave up.

// One product of a launch: its operands' maps and its arguments.
template <class Op>
struct Job {
    using Operator = Op;
    CUtensorMap map_a, map_b;
    typename Op::Args args;
};

// The place of a role in the ring of stages, and of the issuer in the accumulators.
struct Ring {
    uint32_t it, st, phase, n;
    template <class L>
    __device__ __forceinline__ void step() {
        ++it;
        if (++st == static_cast<uint32_t>(L::kStages)) {
            st = 0;
            phase ^= 1u;
        }
    }
};

// A tile's copies, by the producer's warp.
template <class Op>
__device__ __forceinline__ bool produce(const Job<Op>& job, const Shape& s, int unit, int rank, Sync& sy, uint8_t* smem, Ring& r) {
    using L = typename Op::Layout;
    constexpr int P = L::kP;
    const uint64_t pol_a = Op::kAKeep ? policy_evict_last() : policy_evict_first();
    const uint64_t pol_b = Op::kBKeep ? policy_evict_last() : policy_evict_first();
    const Tile t = tile_at(job.args.shape, unit);
    const Shape& o = job.args.shape;
    const int am = o.a_mn + (t.m * P + rank) * kRows, bn = o.b_mn + t.n * L::kTN + rank * L::kBRows, k0 = t.k0 * L::kK;
    for (int k = 0; k < t.steps; ++k) {
        if (r.it >= static_cast<uint32_t>(L::kStages) && !__all_sync(~0u, wait_or_abort(sy, &sy.empty[r.st], r.phase, s))) return false;
        uint8_t* dst = smem + r.st * L::kBytes;
        uint32_t bar;
        if constexpr (P == 1) bar = smem_u32(&sy.full[r.st]);
        else bar = cluster_map(&sy.full[r.st], 0);
        if (elect_one()) {
            if (P == 1 || rank == 0) mbar_arrive_expect_tx(&sy.full[r.st], P * L::kBytes);
            load_operand<L, L::kAMn>(dst, &job.map_a, kRows, am, o.a_k + k0 + k * L::kK, bar, pol_a);
            load_operand<L, L::kBMn>(dst + L::kABytes, &job.map_b, L::kBRows, bn, o.b_k + k0 + k * L::kK, bar, pol_b);
        }
        __syncwarp();
        r.step<L>();
    }
    return true;
}

// A tile's matrix instructions, by an issuer's warp. With an accumulator per step two issuers take
// the steps in turn: one alone takes 500 cycles for a step's waits and instructions, as
// long as they run.
template <class Op>
__device__ __forceinline__ bool issue(const Job<Op>& job, const Shape& s, int unit, int issuer, uint32_t tmem, Sync& sy, uint8_t* smem, Ring& r) {
    using L = typename Op::Layout;
    constexpr int P = L::kP;
    static_assert(L::kIssuers == 1 || Op::kChunk == 1, "one issuer's instructions sum up in order");
    constexpr uint32_t kIdesc = tc::idesc_f(Op::kFormat, L::kAMn, L::kBMn, kRows * P, L::kTN);
    constexpr bool kF8 = L::kElem == 1;
    // 32 bytes of K: along a 128-byte row, or (MN-major) as many whole rows as elements
    constexpr uint32_t kStepA = L::kAMn ? 32 / L::kElem * 128 / 16 : 2, kStepB = L::kBMn ? 32 / L::kElem * 128 / 16 : 2;
    const uint32_t base = smem_u32(smem);
    const uint64_t first_a = L::kAMn ? tc::desc_operand_mn(base, L::kK) : tc::desc_operand(base);
    const uint64_t first_b = L::kBMn ? tc::desc_operand_mn(base + L::kABytes, L::kK) : tc::desc_operand(base + L::kABytes);
    const int steps = tile_at(job.args.shape, unit).steps;
    const auto first_of = [&](int k) {   // whether step k starts an accumulator
        return Op::kChunk == kPerLaunch ? (k & (job.args.shape.chunk - 1)) == 0 : k % (Op::kChunk | (Op::kChunk == 0)) == 0;
    };
    for (int k = 0; k < steps; ++k) {
        if (L::kIssuers > 1 && r.it % L::kIssuers != static_cast<uint32_t>(issuer)) {
            ++r.n;
            r.step<L>();
            continue;
        }
        const uint32_t use = r.n / L::kBuffers, b = r.n % L::kBuffers, d = tmem + b * L::kTN;
        bool ok = wait_or_abort(sy, &sy.full[r.st], r.phase, s);   // the operands have landed,
        if (first_of(k) && use > 0)                                // and the accumulator has been read
            ok = ok && wait_or_abort(sy, &sy.acc_empty[b], (use - 1) & 1, s);
        if (!__all_sync(~0u, ok)) return false;
        tc::fence_after_sync();
        const uint64_t da = first_a + r.st * (L::kBytes / 16), db = first_b + r.st * (L::kBytes / 16);
        const bool begin = first_of(k), last = first_of(k + 1) || k == steps - 1;
        if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::mma_f<P, kF8>(d, da + kStepA * j, db + kStepB * j, kIdesc, !begin || j > 0);
            if (last) tc::commit_all<P>(&sy.acc_full[b]);
            tc::commit_all<P>(&sy.empty[r.st]);
        }
        __syncwarp();
        if (last) ++r.n;
        r.step<L>();
    }
    return true;
}

// Accumulators of a tile.
template <class Op>
__device__ __forceinline__ int chunks_of(const Job<Op>& job, int unit) {
    const Shape& s = job.args.shape;
    return (tile_at(s, unit).steps - 1) / (Op::kChunk == kPerLaunch ? s.chunk : Op::kChunk) + 1;
}

// One product, or two of the same layout sizes that do not depend on one another: the second's
// tiles follow the first's, and fill its last round over the SMs.
template <class Op, class Op2 = void>
struct Jobs {
    using Layout = typename Op::Layout;
    Job<Op> first;
    Job<Op2> second;
    static_assert(Layout::kP == Op2::Layout::kP && Layout::kBytes == Op2::Layout::kBytes && Layout::kTN == Op2::Layout::kTN &&
                  Layout::kEpiWarps == Op2::Layout::kEpiWarps, "one ring for both");
    __host__ __device__ int units() const { return first.args.shape.units() + second.args.shape.units(); }
    // f(job, unit) of the job that this unit belongs to
    template <class F>
    __device__ __forceinline__ auto at(int unit, F f) const {
        const int n = first.args.shape.units();
        return unit < n ? f(first, unit) : f(second, unit - n);
    }
};
template <class Op>
struct Jobs<Op, void> {
    using Layout = typename Op::Layout;
    Job<Op> first;
    __host__ __device__ int units() const { return first.args.shape.units(); }
    template <class F>
    __device__ __forceinline__ auto at(int unit, F f) const {
        return f(first, unit);
    }
};

template <class J>
__global__ void __launch_bounds__(J::Layout::kThreads, 1) product_kernel(const __grid_constant__ J jobs) {
    using L = typename J::Layout;
    constexpr int P = L::kP, kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Sync sy;
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = P == 1 ? 0 : static_cast<int>(cluster_ctarank());
    const Shape& s = jobs.first.args.shape;   // (its error word, limits and self-test are the launch's)
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sy.full[i], 1);
            mbar_init(&sy.empty[i], 1);
        }
        for (int i = 0; i < L::kBuffers; ++i) {
            mbar_init(&sy.acc_full[i], 1);
            mbar_init(&sy.acc_empty[i], L::kEpiWarps + (rank == 0 ? P - 1 : 0));   // rank 0: rank 1's forwarder too
        }
        mbar_init(&sy.issued, L::kIssuers);
        mbar_init_fence();
        sy.abort = 0u;
        sy.copies = 0u;
    }
    __syncwarp();
    if (warp == 0) tc::tmem_alloc_of<P>(&sy.tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (P > 1) {   // the other CTA's barriers are ready too
        cluster_fence();
        cluster_sync_all();
    }
    tc::fence_after_sync();
    programmatic_wait();
    const uint32_t tmem = sy.tmem;
    const int units = jobs.units();
    const int first = static_cast<int>(blockIdx.x) / P, stride = static_cast<int>(gridDim.x) / P;

    // (the producer's and the issuer's warps run their loops whole, one elected lane issues)
    if (warp == L::kProducer && s.idle != kRoleProducer) {
        Ring r = {0, 0, 1, 0};   // the phase of `empty` before the current use of the slot
        for (int i = first; i < units; i += stride)
            if (!jobs.at(i, [&](const auto& job, int unit) { return produce(job, s, unit, rank, sy, smem, r); })) break;
        // The copies in flight land, and the last signals of other CTAs, before the CTAs end,
        // whoever gave up (a pair's copies complete on rank 0's barriers; all bounded).
        for (uint32_t b = r.it > static_cast<uint32_t>(kStages) ? r.it - kStages : 0; b < r.it; ++b) {
            if ((P == 1 || rank == 0) && !mbar_wait(&sy.full[b % kStages], (b / kStages) & 1, kDrainRounds)) break;
            if (P > 1 && !mbar_wait(&sy.empty[b % kStages], (b / kStages) & 1, kDrainRounds)) break;
        }
        if (lane == 0) sy.copies = r.it;
    } else if (warp >= L::kIssuer && (P == 1 || rank == 0) && s.idle != kRoleIssuer) {
        Ring r = {0, 0, 0, 0};
        for (int i = first; i < units; i += stride)
            if (!jobs.at(i, [&](const auto& job, int unit) { return issue(job, s, unit, warp - L::kIssuer, tmem, sy, smem, r); })) break;
        // the issued instructions finish before tensor memory is freed, whoever gave up (bounded)
        if (elect_one()) tc::commit_own<P>(&sy.issued);
        __syncwarp();
        mbar_wait(&sy.issued, 0, kDrainRounds);
    } else if (P > 1 && warp == L::kIssuer && lane == 0 && rank == 1 && s.idle != kRoleIssuer) {
        // rank 1's forwarder: its CTA has read an accumulator (one arrival from another CTA, in
        // place of one per warp)
        uint32_t n = 0;
        bool ok = true;
        for (int i = first; ok && i < units; i += stride)
            for (int u = jobs.at(i, [&](const auto& job, int unit) { return chunks_of(job, unit); }); ok && u > 0; --u, ++n)
                if ((ok = wait_or_abort(sy, &sy.acc_empty[n % L::kBuffers], (n / L::kBuffers) & 1, s))) arrive_rank0(&sy.acc_empty[n % L::kBuffers]);
    } else if (warp < L::kEpiWarps && s.idle != kRoleEpilogue) {
        Acc<L> acc(sy, s, tmem);
        for (int i = first; i < units; i += stride)
            if (!jobs.at(i, [&](const auto& job, int unit) {
                    return std::decay_t<decltype(job)>::Operator::tile(job.args, tile_at(job.args.shape, unit), warp, lane, rank, acc);
                }))
                break;
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if constexpr (P > 1) {   // neither CTA ends while the other still reads or signals it
        cluster_fence();
        cluster_sync_all();
    }
    tc::fence_after_sync();
    if (s.idle >= 0 && (P == 1 || rank == 0) && threadIdx.x == 0) {   // the self-test: nothing of this tile's is in flight
        bool done = s.idle == kRoleIssuer || mbar_test(&sy.issued, 0);
        for (uint32_t i = 0; i < static_cast<uint32_t>(kStages) && i < sy.copies; ++i)   // the last use of slot i
            done = mbar_test(&sy.full[i], ((sy.copies - 1 - i) / kStages) & 1) && done;
        if (!done && s.error != nullptr) atomicOr(s.error, kDevErrUnfinished);
    }
    if (warp == 0) tc::tmem_free_of<P>(tmem, 512);
}

// ------------------------------------------------------------------- host ----

// Launches in clusters of `ctas`, allowed to start (up to its programmatic_wait) while the kernel
// before it on the stream finishes.
template <class... Params, class... Given>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, int ctas, cudaStream_t stream, Given&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Given>(args)...);
}

inline Shape whole_tiles(int tiles_m, int tiles_n, int steps, unsigned int* error) {
    Shape s = {};
    s.tiles_m = tiles_m;
    s.tiles_n = tiles_n;
    s.whole = tiles_m * tiles_n;
    s.splits = 1;
    s.steps = s.split_steps = steps;
    s.error = error;
    return s;
}

// A tensor map of a row-major matrix: `rows` rows of `cols` elements, `ld` bytes apart, read in
// boxes of 128 bytes by box_rows with the 128-byte swizzle; what lies outside reads as zeros.
// base and ld: multiples of 16 bytes.
cudaError_t encode_map(CUtensorMap* map, const void* base, int elem, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows);

// The maps of an operand of `Layout` L: K-major, mn rows of k elements; MN-major, k rows of mn.
template <class L, bool MN>
cudaError_t encode_operand(CUtensorMap* map, const void* base, uint64_t mn, uint64_t k, uint64_t ld_bytes, int box_mn) {
    return MN ? encode_map(map, base, L::kElem, mn, k, ld_bytes, L::kK) : encode_map(map, base, L::kElem, k, mn, ld_bytes, box_mn);
}

template <class J>
cudaError_t launch(J& jobs, cudaStream_t stream) {
    using L = typename J::Layout;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    constexpr int kDevices = 64;
    static std::atomic<bool> known[kDevices];   // per device: the kernel's shared memory has been allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(product_kernel<J>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
        if (e != cudaSuccess) return e;
        known[dev].store(true, std::memory_order_release);
    }
    Shape& s = jobs.first.args.shape;
    if (s.rounds == 0) {
        s.rounds = kWaitLimit / kWaitSlices;
        s.idle = -1;
    }
    const int units = jobs.units(), most = sms / L::kP;
    return launch_early(product_kernel<J>, dim3(static_cast<unsigned>((units < most ? units : most) * L::kP)), L::kThreads, L::kSmem, L::kP, stream, jobs);
}

}  // namespace gemm
}  // namespace dh
