// The FP8 block-scaled product (dh_fp8_blocks.cu) for up to 64 tokens, where reading the weight
// is the work: rows of the weight lie along the rows of a tile (128 of them), the tokens along
// its 16 to 64 columns, so that the matrix instructions waste nothing on tokens that are not
// there, and a step of 128 features is one 16 KB box of the weight.
//
// To have every SM read, the contraction is split over the CTAs of a cluster (1 to 8): each sums
// its steps in registers, then sends each token's sums to the CTA that stores that token,
// through distributed shared memory; sums are joined in the order of the ranks. Where
// they are few the activations are quantised in the kernel too, by each CTA for its own steps,
// while its first boxes of the weight are on their way: one launch in all.
//
// What bounds it: reading the weight where that is long (the head of 64,026 x 2,560 at 1 token 30 us,
// 5.4 TB/s, at 32 tokens 33: 501 tiles make four rounds over 152 SMs, the last of them of 45), else
// the chain of a launch, a ring of boxes, the exchange and the stores (1 x 4,608 x 2,560 6.1 us,
// 16 x 2,560 x 5,120 9.1; tokens along the rows, in one part, 26.7 and 46).
#pragma once

#include "dh_fp8_blocks.cuh"

namespace dh {
namespace f8 {

using gemm::ceil_div;

constexpr int kEpiWarps = 8, kProducer = kEpiWarps, kIssuer = kProducer + 1, kThreads = 32 * (kIssuer + 1);
constexpr int kBuffers = 4;                       // accumulators in tensor memory
constexpr int kABytes = kBlock * kBlock;          // a step's box of the weight
constexpr int kSpace = 224 * 1024;                // shared memory for stages, codes, scales and exchange
constexpr int kMaxSplits = 8;

struct FewArgs {
    const void* x;            // quantised here: [M][width]
    long long ldx;
    int width, vec;           // vec: its rows are 16-byte aligned
    const float* scales;      // else [steps][M]
    const float* sw;          // scale of output block j and step b at j * sw_j + b * sw_b
    int sw_j, sw_b;
    int M, N;                 // tokens, output features
    int tiles, steps, per;    // tiles of 128 outputs; steps in all and per CTA of a cluster
    int stages;
    void* y;
    long long ldy;
    unsigned int* error;
    uint32_t rounds;          // tries of a bounded wait, times kWaitSlices
    int idle;                 // self-test: the role that does nothing (-1: none)
};

struct FewSync {
    uint64_t full[16], empty[16], acc_full[kBuffers], acc_empty[kBuffers], codes, received, room, issued;
    uint32_t tmem;
    unsigned int abort;
    uint32_t copies;   // self-test: stages that the producer filled
};

__device__ __forceinline__ bool wait(FewSync& sy, uint64_t* bar, uint32_t parity, const FewArgs& a) {
    return mbar_wait<false>(bar, parity, 1) || gemm::wait_longer(&sy.abort, bar, parity, a.rounds, a.error);
}
// The same for a barrier that other CTAs of the cluster arrive on: their writes are visible after it.
__device__ __forceinline__ bool wait_cluster(FewSync& sy, uint64_t* bar, uint32_t parity, const FewArgs& a) {
    for (int i = 0; i < gemm::kWaitSlices; ++i) {
        if (mbar_wait_cluster(bar, parity, a.rounds)) return true;
        if (*const_cast<volatile unsigned int*>(&sy.abort) != 0u) return false;
    }
    *const_cast<volatile unsigned int*>(&sy.abort) = 1u;
    if (a.error != nullptr) atomicOr(a.error, kDevErrTimeout);
    return false;
}

template <int NT, bool FUSED>
struct Few {
    static constexpr int kPart = NT / 2;                                 // tokens of an epilogue warp
    static constexpr int kStage = kABytes + (FUSED ? 0 : NT * kBlock);
    static constexpr int kCols = kBuffers * NT < 32 ? 32 : kBuffers * NT;
    // Shared memory besides the stages for CTAs of `per` steps in clusters of `splits`.
    __host__ __device__ static constexpr int rest(int per, int splits) {
        return (FUSED ? per * NT * kBlock : 0) + (per * NT * 4 + 1023) / 1024 * 1024 + (splits > 1 ? splits * ((NT + splits - 1) / splits) * kBlock * 4 : 0);
    }
};

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[N]) {
    if constexpr (N == 8) tc::tmem_load8(at, r);
    else if constexpr (N == 16) tc::tmem_load16(at, r);
    else tc::tmem_load32(at, r);
}

template <class TX, class TY, int NT, bool FUSED, bool GRADIENT>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ CUtensorMap map_w,
                                                          const __grid_constant__ CUtensorMap map_x, const FewArgs a) {
    using F = Few<NT, FUSED>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ FewSync sy;
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int splits = ceil_div(a.steps, a.per), rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = static_cast<int>(blockIdx.x) / splits, stride = static_cast<int>(gridDim.x) / splits;
    const int b0 = rank * a.per, count = min(a.per, a.steps - b0);
    uint8_t* codes = smem + a.stages * F::kStage;                        // FUSED: [count][NT][128]
    float* scales = reinterpret_cast<float*>(codes + (FUSED ? a.per * NT * kBlock : 0));   // [count][NT]
    float* exchange = scales + (a.per * NT * 4 + 1023) / 1024 * 256;     // [rank][ceil(NT / splits)][128]
    const uint32_t stages = static_cast<uint32_t>(a.stages);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&sy.full[i], 1);
            mbar_init(&sy.empty[i], 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&sy.acc_full[i], 1);
            mbar_init(&sy.acc_empty[i], kEpiWarps);
        }
        mbar_init(&sy.codes, 32 * kEpiWarps);
        mbar_init(&sy.received, kEpiWarps * splits);
        mbar_init(&sy.room, kEpiWarps * splits);
        mbar_init(&sy.issued, 1);
        mbar_init_fence();
        sy.abort = 0u;
        sy.copies = 0u;
    }
    __syncwarp();
    if (warp == kIssuer) tc::tmem_alloc(&sy.tmem, F::kCols);
    tc::fence_before_sync();
    __syncthreads();
    // The other CTAs' barriers are ready before the first exchange: arrived here, waited for there
    // (and by the producer and the issuer at their ends).
    if (splits > 1) {
        cluster_fence();
        cluster_arrive();
    }
    tc::fence_after_sync();
    programmatic_wait();
    const uint32_t tmem = sy.tmem;

    if (warp == kProducer) {
        uint64_t policy;
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        uint32_t it = 0, st = 0, phase = 1;
        bool ok = a.idle != gemm::kRoleProducer;
        for (int t = first; ok && t < a.tiles; t += stride)
            for (int b = b0; b < b0 + count; ++b, ++it) {
                if (it >= stages && !(ok = __all_sync(~0u, wait(sy, &sy.empty[st], phase, a)))) break;
                uint8_t* dst = smem + st * F::kStage;
                const uint32_t bar = smem_u32(&sy.full[st]);
                if (gemm::elect_one()) {
                    mbar_arrive_expect_tx(&sy.full[st], F::kStage);
                    gemm::tma_2d<1>(dst, &map_w, GRADIENT ? t * kBlock : b * kBlock, GRADIENT ? b * kBlock : t * kBlock, bar, policy);
                    if (!FUSED) gemm::tma_2d<1>(dst + kABytes, &map_x, b * kBlock, 0, bar, policy);
                }
                __syncwarp();
                if (++st == stages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        // the copies in flight land before the CTA ends, whoever gave up (bounded)
        for (uint32_t b = it > stages ? it - stages : 0; b < it; ++b)
            if (!mbar_wait(&sy.full[b % stages], (b / stages) & 1, gemm::kDrainRounds)) break;
        if (lane == 0) sy.copies = it;
        __syncwarp();
        if (splits > 1) cluster_wait();
    } else if (warp == kIssuer) {
        constexpr uint32_t kIdesc = tc::idesc_f(0, GRADIENT, false, kBlock, NT), kStepA = GRADIENT ? 256 : 2;
        const uint32_t base = smem_u32(smem);
        const uint64_t first_a = GRADIENT ? tc::desc_operand_mn(base, kBlock) : tc::desc_operand(base);
        const uint64_t first_b = tc::desc_operand(FUSED ? smem_u32(codes) : base + kABytes);
        uint32_t n = 0, st = 0, phase = 0;
        bool ok = a.idle != gemm::kRoleIssuer && (!FUSED || __all_sync(~0u, wait(sy, &sy.codes, 0, a)));
        for (int t = first; ok && t < a.tiles; t += stride)
            for (int b = 0; b < count; ++b, ++n) {
                const uint32_t buf = n % kBuffers, use = n / kBuffers;
                ok = wait(sy, &sy.full[st], phase, a) && (use == 0 || wait(sy, &sy.acc_empty[buf], (use - 1) & 1, a));
                if (!(ok = __all_sync(~0u, ok))) break;
                tc::fence_after_sync();
                const uint64_t da = first_a + st * (F::kStage / 16), db = first_b + (FUSED ? b * (NT * kBlock / 16) : st * (F::kStage / 16));
                if (gemm::elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) tc::mma_f<1, true>(tmem + buf * NT, da + kStepA * j, db + 2 * j, kIdesc, j > 0);
                    tc::commit(&sy.acc_full[buf]);
                    tc::commit(&sy.empty[st]);
                }
                __syncwarp();
                if (++st == stages) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        if (gemm::elect_one()) tc::commit(&sy.issued);
        __syncwarp();
        mbar_wait(&sy.issued, 0, gemm::kDrainRounds);
        __syncwarp();
        if (splits > 1) cluster_wait();
    } else {
        if (FUSED) {   // eight lanes per token and step
            const Rows<TX> x = {static_cast<const TX*>(a.x), a.ldx, a.M, a.width};
#pragma unroll 2
            for (int u0 = warp * 4; u0 < a.M * count; u0 += 4 * kEpiWarps) {
                const int u = u0 + (lane >> 3), m = u % a.M, b = u / a.M, k = (b0 + b) * kBlock + (lane & 7) * 16;
                const int n = b < count ? min(16, a.width - k) : 0;
                uint4 w;
                const float s = a.vec ? encode16<TX, true>(x, m, k, n, w) : encode16<TX, false>(x, m, k, n, w);
                if (b < count) {
                    *reinterpret_cast<uint4*>(codes + (b * NT + m) * kBlock + (((lane & 7) ^ (m & 7)) << 4)) = w;
                    if ((lane & 7) == 0) scales[b * NT + m] = s;
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive(&sy.codes);
        } else {
            for (int i = threadIdx.x; i < count * NT; i += 32 * kEpiWarps) {
                const int m = i % NT, b = i / NT;
                scales[i] = m < a.M ? a.scales[static_cast<size_t>(b0 + b) * a.M + m] : 0.0f;
            }
        }
        named_bar_sync(1, 32 * kEpiWarps);   // the scales are there for every warp
        const int quarter = warp & 3, part = warp >> 2, local = quarter * 32 + lane;
        uint32_t n = 0, e = 0;
        bool joined = splits == 1;   // the cluster's start has been waited for
        for (int t = a.idle != gemm::kRoleEpilogue ? first : a.tiles; t < a.tiles; t += stride, ++e) {
            const int row = t * kBlock + local;
            const float* sw = a.sw + static_cast<size_t>(t) * a.sw_j + static_cast<size_t>(b0) * a.sw_b;
            float next = __ldg(sw);
            float sum[F::kPart];
#pragma unroll
            for (int i = 0; i < F::kPart; ++i) sum[i] = 0.0f;
            bool ok = true;
#pragma unroll 1
            for (int b = 0; b < count; ++b, ++n) {
                const float w = next;
                if (b + 1 < count) next = __ldg(sw + static_cast<size_t>(b + 1) * a.sw_b);
                const uint32_t buf = n % kBuffers;
                if (!(ok = __all_sync(~0u, wait(sy, &sy.acc_full[buf], (n / kBuffers) & 1, a)))) break;
                tc::fence_after_sync();
                const uint32_t from = tmem + (static_cast<uint32_t>(quarter) << 21) + buf * NT + part * F::kPart;
                const float4* sx = reinterpret_cast<const float4*>(scales + b * NT + part * F::kPart);
                constexpr int kLoad = F::kPart < 32 ? F::kPart : 32;
#pragma unroll
                for (int c = 0; c < F::kPart; c += kLoad) {
                    uint32_t r[kLoad];
                    tmem_load(from + c, r);
                    tc::tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < kLoad; i += 4) {
                        const float4 s = sx[(c + i) / 4];
                        sum[c + i] = fmaf(s.x * w, __uint_as_float(r[i]), sum[c + i]);
                        sum[c + i + 1] = fmaf(s.y * w, __uint_as_float(r[i + 1]), sum[c + i + 1]);
                        sum[c + i + 2] = fmaf(s.z * w, __uint_as_float(r[i + 2]), sum[c + i + 2]);
                        sum[c + i + 3] = fmaf(s.w * w, __uint_as_float(r[i + 3]), sum[c + i + 3]);
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sy.acc_empty[buf]);
            }
            if (!ok) break;
            TY* y = static_cast<TY*>(a.y) + row;
            if (splits == 1) {
                if (row < a.N) {
#pragma unroll
                    for (int i = 0; i < F::kPart; ++i) {
                        const int m = part * F::kPart + i;
                        if (m < a.M) y[static_cast<size_t>(m) * a.ldy] = dh::rows::Elem<TY>::store(sum[i]);
                    }
                }
                __syncwarp();
                continue;
            }
            if (!joined) cluster_wait();
            joined = true;
            // token m to rank m % splits; what the others sent last has been read everywhere first
            if (e > 0 && !__all_sync(~0u, wait_cluster(sy, &sy.room, (e - 1) & 1, a))) break;
            const int slots = (NT + splits - 1) / splits;
#pragma unroll
            for (int i = 0; i < F::kPart; ++i) {
                const int m = part * F::kPart + i;
                if (m < a.M) st_cluster_f32(cluster_map(exchange + (rank * slots + m / splits) * kBlock + local, m % splits), sum[i]);
            }
            __syncwarp();
            if (lane < splits) mbar_arrive_remote(cluster_map(&sy.received, lane));
            __syncwarp();
            if (!__all_sync(~0u, wait_cluster(sy, &sy.received, e & 1, a))) break;
            for (int slot = part; slot * splits + rank < a.M; slot += 2) {
                float v = exchange[slot * kBlock + local];
                for (int r = 1; r < splits; ++r) v += exchange[(r * slots + slot) * kBlock + local];
                if (row < a.N) y[static_cast<size_t>(slot * splits + rank) * a.ldy] = dh::rows::Elem<TY>::store(v);
            }
            __syncwarp();
            if (lane < splits) mbar_arrive_remote(cluster_map(&sy.room, lane));
            __syncwarp();
        }
        if (!joined) cluster_wait();
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (splits > 1) {   // no CTA ends while another may still write to it
        cluster_fence();
        cluster_sync_all();
    }
    tc::fence_after_sync();
    if (a.idle >= 0 && threadIdx.x == 0) {   // the self-test: nothing of this CTA's is in flight
        bool done = mbar_test(&sy.issued, 0);
        for (uint32_t i = 0; i < stages && i < sy.copies; ++i) done = mbar_test(&sy.full[i], ((sy.copies - 1 - i) / stages) & 1) && done;
        if (!done && a.error != nullptr) atomicOr(a.error, kDevErrUnfinished);
    }
    if (warp == kIssuer) tc::tmem_free(tmem, F::kCols);
}

// ------------------------------------------------------------------- host ----

// Clusters of 1 to 8 CTAs of this memory that run at once (they do not span the GPU's processing
// clusters).
constexpr int kClusters[kMaxSplits + 1] = {0, kSms, kSms / 2, 46, 36, 28, 23, 15, 15};

template <class TX, class TY, int NT, bool FUSED, bool GRADIENT>
cudaError_t launch_kernel(const CUtensorMap& map_w, const CUtensorMap& map_x, FewArgs a, int splits, cudaStream_t stream) {
    using F = Few<NT, FUSED>;
    constexpr auto kernel = few_kernel<TX, TY, NT, FUSED, GRADIENT>;
    constexpr int kDevices = 64, kSmem = kSpace + 1024;
    static std::atomic<bool> known[kDevices];   // per device: the kernel's shared memory has been allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
        known[dev].store(true, std::memory_order_release);
    }
    const int fit = (kSpace - F::rest(a.per, splits)) / F::kStage;
    a.stages = fit < 16 ? fit : 16;
    const int want = a.tiles < kClusters[splits] ? a.tiles : kClusters[splits];
    return gemm::launch_early(kernel, dim3(static_cast<unsigned>(want * splits)), kThreads, kSmem, splits, stream, map_w, map_x, a);
}

template <class TX, class TY, int NT, bool FUSED>
cudaError_t launch_sized(const Fp8BlockArgs& f, int splits, const uint8_t* codes, int ldc, const float* scales, cudaStream_t s) {
    const int width = f.gradient ? f.N : f.K, out = f.gradient ? f.K : f.N, kb = ceil_div(f.K, kBlock);
    FewArgs a = {};
    a.x = f.x;
    a.ldx = f.ldx;
    a.width = width;
    a.vec = rows_aligned16(f.x, f.ldx * static_cast<long long>(sizeof(TX)), f.M);
    a.scales = scales;
    a.sw = f.scale;
    a.sw_j = f.gradient ? 1 : kb;
    a.sw_b = f.gradient ? kb : 1;
    a.M = f.M;
    a.N = out;
    a.tiles = ceil_div(out, kBlock);
    a.steps = ceil_div(width, kBlock);
    a.y = f.y;
    a.ldy = f.ldy;
    a.error = f.error;
    a.rounds = f.probe_rounds != 0 ? f.probe_rounds : kWaitLimit / gemm::kWaitSlices;
    a.idle = f.probe_rounds != 0 ? f.probe_role : -1;
    a.per = ceil_div(a.steps, splits);
    CUtensorMap map_w, map_x;
    // (the same box either way: 128 bytes of a row of W by 128 rows)
    cudaError_t e = gemm::encode_map(&map_w, f.q, 1, f.K, f.N, f.K, kBlock);
    if (e != cudaSuccess) return e;
    if (FUSED) map_x = map_w;
    else if ((e = gemm::encode_map(&map_x, codes, 1, width, f.M, ldc, NT)) != cudaSuccess) return e;
    return f.gradient ? launch_kernel<TX, TY, NT, FUSED, true>(map_w, map_x, a, splits, s)
                      : launch_kernel<TX, TY, NT, FUSED, false>(map_w, map_x, a, splits, s);
}

template <class TX, class TY>
cudaError_t launch_fused(const Fp8BlockArgs& f, const FewPlan& p, cudaStream_t s) {
    return p.columns == 16   ? launch_sized<TX, TY, 16, true>(f, p.splits, nullptr, 0, nullptr, s)
           : p.columns == 32 ? launch_sized<TX, TY, 32, true>(f, p.splits, nullptr, 0, nullptr, s)
                             : launch_sized<TX, TY, 64, true>(f, p.splits, nullptr, 0, nullptr, s);
}

template <class TY>
cudaError_t launch_few(const Fp8BlockArgs& f, const FewPlan& p, const uint8_t* codes, int ldc, const float* scales, cudaStream_t s) {
    if (p.fused)
        return f.x_type == DH_T_BF16  ? launch_fused<__nv_bfloat16, TY>(f, p, s)
               : f.x_type == DH_T_F16 ? launch_fused<__half, TY>(f, p, s)
                                      : launch_fused<float, TY>(f, p, s);
    // (the element type of x matters to the fused form alone)
    return p.columns == 32 ? launch_sized<float, TY, 32, false>(f, p.splits, codes, ldc, scales, s)
                           : launch_sized<float, TY, 64, false>(f, p.splits, codes, ldc, scales, s);
}

}  // namespace f8
}  // namespace dh
