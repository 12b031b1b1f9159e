// NVFP4 x NVFP4 product of many tokens (W4A4): y = x W'^T with the activations
// quantised to NVFP4 per token on the fly.
//
//   g_m = max(max_k |x_mk|, 1e-12) / 2688,  s = E4M3_RNE(bamax / (6 g_m)) per
//   block of 16, code = E2M1_RNE(clamp(x / fp32(dec(s) g_m), +-6)): the weights'
//   recipe (dh_quantize.cu) with one global scale per token, so a token's
//   result does not depend on the others in the batch;
//   y_mn = g g_m sum_blocks s_mb s_nb sum_16 c_mk c_nk, accumulated in 32 bits.
//
// Operand layout ("blocks"): 128 rows x 256 k = 16,384 bytes of codes (rows of
// 128 bytes, 16-byte pieces of row r permuted by XOR with r % 8: the 128-byte
// swizzle that the tensor core reads) followed by 2,048 bytes of scales (for
// each 64-wide k-step 512 bytes, [row % 32][row / 32][4 blocks]: the order in
// which one copy moves them to tensor memory). Blocks are ordered [rows / 128]
// [k / 256], rows and k padded with zeros, so a tile's operands for one k-stage are
// contiguous and move with plain bulk copies; no tensor map is needed. Weights are
// packed once (nvfp4_pack_matmul); the activations' quantiser writes its codes
// straight into blocks.
//
// Product kernel: persistent, one CTA per SM; output tiles of 128 tokens x TN
// weight rows. One thread streams blocks into a ring of shared-memory stages;
// four warps, one per group of 32 lanes of tensor memory, move a stage's scales
// there through registers, two such groups in turn; one thread issues the matrix instructions
// (kind::mxf4nvf4, block 16); sixteen warps read a tile's accumulators into
// registers, scaled and rounded, free them for the next tile and store.
//
// Bound, 8,192 tokens on a 64,064 x 2,560 head (567 us with the quantiser's 20:
// 4.8 PFLOP/s; 1.05 GB of results alone take 155 us at the measured copy rate): a
// stage's way through the ring; no unit is saturated. A 128 x 256 x 256 step takes
// 515 ns, 270 of them matrix instructions (64 of k each; the 96-wide ones of sm_103a,
// nominally half as fast again, are not used); it moves 55 KB into shared memory and reads 72 KB there (48 for
// the matrix instructions, 24 for the scales: each of four warps reads them all), 122
// bytes a cycle, half of the banks' peak. 47 bytes a cycle enter an SM from L2, 37 of 100
// that its port takes (2,048 x 32,000 x 2,560: 13.7 TB/s over the GPU). Tiles of 256 x 192 move a fifth less from
// L2, but have room for three stages: 583 against 594, each with one group of scale
// warps (three slots do not go round between two).
// What the choices measured there:
//  - scales: tcgen05.cp takes its turn among the matrix instructions (24 ns a copy,
//    12 copies against 270 ns of matrix instructions per stage); stored from
//    registers while the stages before multiply: 1,067 -> 703 us (with eight
//    epilogue warps that free the accumulators before they store, not four after);
//  - sixteen epilogue warps (a shorter read of the single accumulator buffer): 653;
//  - results stored past L1, whose data array the ring shares: 620; both operands
//    kept in L2 against the results (evict_last): 600; the producer's pointers and
//    phases running along: 590; two groups of scale warps in turn (fewer held results
//    for the registers): 567. 100 tokens: weights, read once, not kept 26.7 -> 24.6;
//  - pairs of CTAs on one 256 x 256 tile (cta_group::2) need a third less of the
//    operands, but each ring slot's round trip crosses the pair twice: 913, with the
//    scales through registers 1,021; operands multicast in clusters of four and
//    eight 971 to 1,163; blocks of 128 k, twice as many stages of half the size, 763;
//    the tokens' scales by tcgen05.cp, the weights' through registers 609; four groups
//    of scale warps beside eight epilogue warps 572.
#include <atomic>
#include <cfloat>

#include "../../include/drafthead.h"
#include "dh_internal.h"
#include "dh_rows.cuh"
#include "dh_tcgen05.cuh"

namespace dh {
namespace mm {

constexpr int kRows = 128;                       // rows of a block
constexpr int kStageK = 256;                     // k of a block
constexpr int kCodes = kRows * kStageK / 2;      // 16,384
constexpr int kScales = kRows * kStageK / 16;    // 2,048
constexpr int kBlock = kCodes + kScales;         // 18,432

__host__ __device__ inline int blocks_of(int n, int per) { return (n + per - 1) / per; }

// Byte offsets inside a block: 16-byte piece p (32 codes) of row r, and the
// scale of its 16-element block b (0..15).
__device__ __forceinline__ int code_offset(int r, int p) { return r * 128 + ((p ^ (r & 7)) << 4); }
__device__ __forceinline__ int scale_offset(int r, int b) {
    return kCodes + (b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3);
}

// ---------------------------------------------------------------- packing ----

// One thread per (row, 32-wide piece): its codes and two scales, zeros beyond
// N rows or K columns (K % 16 == 0).
__global__ void pack_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ sf, int N, int K, uint8_t* __restrict__ out) {
    const int nk = blocks_of(K, kStageK), per_row = nk * (kStageK / 32);
    const size_t total = static_cast<size_t>(blocks_of(N, kRows)) * kRows * per_row;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
         i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const size_t row = i / per_row;
        const int piece = static_cast<int>(i % per_row);
        uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
        uint32_t s0 = 0, s1 = 0;
        const int k = piece * 32;
        if (row < static_cast<size_t>(N)) {
            const uint8_t* src = q + row * (K / 2) + k / 2;
            const uint8_t* s = sf + row * (K / 16) + k / 16;
            if (k < K) {
                lo = *reinterpret_cast<const uint2*>(src);
                s0 = s[0];
            }
            if (k + 16 < K) {
                hi = *reinterpret_cast<const uint2*>(src + 8);
                s1 = s[1];
            }
        }
        uint8_t* blk = out + ((row / kRows) * nk + piece / 8) * kBlock;
        const int r = static_cast<int>(row % kRows), p = piece % 8;
        *reinterpret_cast<uint4*>(blk + code_offset(r, p)) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        *reinterpret_cast<uint16_t*>(blk + scale_offset(r, 2 * p)) = static_cast<uint16_t>(s0 | (s1 << 8));
    }
}

// ------------------------------------------------------------ quantisation ----

constexpr int kQThreads = 128;

__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 elements at p (alignment of the element type only when !VEC), as floats.
template <class T, bool VEC>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
    if constexpr (VEC) {
        constexpr int kVec = rows::Elem<T>::kVec;
#pragma unroll
        for (int i = 0; i < 16 / kVec; ++i)
            rows::Elem<T>::unpack(*reinterpret_cast<const uint4*>(p + i * kVec), reinterpret_cast<float(&)[kVec]>(x[i * kVec]));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = rows::Elem<T>::load(p + i);
    }
}

// One CTA per token: the row's largest magnitude (as bits, so that NaN and
// infinities come out on top), then codes and scales, one 32-wide piece per thread.
// A row with a value that is not finite gets the scale NaN and zero codes:
// its whole result is NaN. Bound by latency: 3 us for 100 rows of 2,560, 20 us for
// 8,192 (42 MB read, 12 written: 2.7 TB/s; the second reading comes from L1). Rows
// held in registers between the two readings cost occupancy: 21.5 us.
template <class T, bool VEC>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const T* __restrict__ x, long long ldx, int K, uint8_t* __restrict__ out,
                                                             float* __restrict__ scale) {
    const int m = blockIdx.x, nk = blocks_of(K, kStageK), nb = K / 16;
    const T* row = x + static_cast<size_t>(m) * ldx;
    uint32_t top = 0;
    for (int b = threadIdx.x; b < nb; b += kQThreads) {
        float v[16];
        load16<T, VEC>(row + b * 16, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    __shared__ uint32_t s_top[kQThreads / 32];
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
    top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    const bool finite = top < 0x7F800000u;
    const float g = finite ? __fdiv_rn(fmaxf(__uint_as_float(top), 1e-12f), 2688.0f) : __uint_as_float(0x7FC00000u);
    const float den = __fmul_rn(6.0f, g);
    if (threadIdx.x == 0) scale[m] = g;
    uint8_t* blk0 = out + static_cast<size_t>(m / kRows) * nk * kBlock;
    const int r = m % kRows;
    for (int piece = threadIdx.x; piece < nk * 8; piece += kQThreads) {
        uint32_t code[4] = {0, 0, 0, 0}, sc[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int b = piece * 2 + h;
            if (b >= nb || !finite) continue;
            float v[16];
            load16<T, VEC>(row + b * 16, v);
            float bmax = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) bmax = fmaxf(bmax, fabsf(v[i]));
            sc[h] = static_cast<uint32_t>(__nv_cvt_float_to_fp8(__fdiv_rn(bmax, den), __NV_SATFINITE, __NV_E4M3));
            const float d = __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(sc[h]), __NV_E4M3))), g);
            if (d == 0.0f) continue;   // zeros (their sign does not matter to a sum of products)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                code[2 * h + i / 4] |= e2m1x2(__fdiv_rn(v[2 * i], d), __fdiv_rn(v[2 * i + 1], d)) << (8 * (i % 4));
        }
        uint8_t* blk = blk0 + static_cast<size_t>(piece / 8) * kBlock;
        *reinterpret_cast<uint4*>(blk + code_offset(r, piece % 8)) = make_uint4(code[0], code[1], code[2], code[3]);
        *reinterpret_cast<uint16_t*>(blk + scale_offset(r, 2 * (piece % 8))) = static_cast<uint16_t>(sc[0] | (sc[1] << 8));
    }
}

// ----------------------------------------------------------------- product ----

struct Args {
    const uint8_t* a;       // activation blocks
    const uint8_t* b;       // weight blocks
    const float* ga;        // [M] token scales
    const float* gb;        // weight scale
    void* y;
    long long ldy;
    int M, N, nk;           // nk: k-stages
    int tiles_m, tiles_n;
    unsigned int* error;    // DH_DEVERR_* word or null
    int idle;               // self-test: the role that does nothing
    uint32_t rounds;        // self-test: tries of a wait, times kWaitSlices
};

// Roles of the warps: a bounded wait tries kWaitSlices times kWaitLimit / kWaitSlices rounds.
enum Role { kRoleProducer, kRoleScales, kRoleIssuer, kRoleEpilogue };
constexpr int kWaitSlices = 64;
constexpr uint32_t kDrainRounds = kWaitLimit / kWaitSlices;   // for a role's own work in flight

// Warps: epilogue, groups of scale warps that take the stages in turn, producer, issuer.
constexpr int kEpiWarps = 16, kSfWarps = 4, kSfGroups = 2, kProducer = kEpiWarps + kSfGroups * kSfWarps, kIssuer = kProducer + 1;
constexpr int kThreads = 32 * (kIssuer + 1);

template <int TN>
struct Cfg {
    static constexpr int kNB = TN / kRows;                        // weight blocks per tile
    // a stage: the token block, the codes of the weight blocks, their scales
    static constexpr int kB = kBlock, kSf = kBlock + kNB * kCodes, kStageBytes = kSf + kNB * kScales;
    static constexpr int kStages = (227 * 1024 - 1024 - 512) / kStageBytes;   // 227 KB less alignment and barriers
    static constexpr int kSmem = kStages * kStageBytes + 1024;    // + alignment to 1,024
    // tensor-memory columns: accumulators (of two tiles where they fit), then every stage's
    // scales (16 of A, 16 per block of B)
    static constexpr int kAcc = TN == 128 ? 2 : 1;
    static constexpr int kSfA = kAcc * TN, kSfB = kSfA + 16, kSfStep = 16 + 16 * kNB;
    static constexpr int kCols = 512;
    static_assert(kSfA + kStages * kSfStep <= kCols, "tensor memory");
    static_assert(kStages <= 8 && kStageBytes % 1024 == 0, "stage layout");
    // A group of scale warps waits for a slot's phases by their parity, so it has to have
    // seen the one before: every use of a slot is the same group's (stages may land out
    // of order).
    static_assert(kStages % kSfGroups == 0, "scale groups");
};

struct Sync {
    uint64_t full[8], empty[8], sf_full[8], acc_full[2], acc_empty[2], issued;
    uint32_t tmem;
    unsigned int abort;
    uint32_t copies;   // self-test: stages that the producer filled
};

// A bounded wait that gives up at once when another role has.
template <bool PROBE>
__device__ __forceinline__ bool wait_or_abort(Sync& sy, uint64_t* bar, uint32_t parity, const Args& a) {
    if (mbar_test(bar, parity)) return true;
    for (int i = 0; i < kWaitSlices; ++i) {
        if (mbar_wait(bar, parity, PROBE ? a.rounds : kWaitLimit / kWaitSlices)) return true;
        if (*const_cast<volatile unsigned int*>(&sy.abort) != 0u) return false;
    }
    *const_cast<volatile unsigned int*>(&sy.abort) = 1u;
    if (a.error != nullptr) atomicOr(a.error, kDevErrTimeout);
    return false;
}

__device__ __forceinline__ void lds16(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}

// 32 bytes, 32-byte aligned, in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
}

// PROBE: the self-test of the waits (nvfp4_matmul_wait_probe): the role a.idle does
// nothing, waits are short, and work still in flight at the end is recorded.
template <class TY, int TN, bool PROBE>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const Args a) {
    using C = Cfg<TN>;
    constexpr int kStages = C::kStages, kCols = TN * 4 / kEpiWarps;   // columns per epilogue warp
    extern __shared__ uint8_t smem_raw[];
    __shared__ Sync sy;
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sy.full[i], 1);
            mbar_init(&sy.empty[i], 1);
            mbar_init(&sy.sf_full[i], kSfWarps);
        }
        for (int i = 0; i < C::kAcc; ++i) {
            mbar_init(&sy.acc_full[i], 1);
            mbar_init(&sy.acc_empty[i], kEpiWarps);
        }
        mbar_init(&sy.issued, 1);
        mbar_init_fence();
        sy.abort = 0u;
        sy.copies = 0u;
    }
    __syncwarp();
    if (warp == 0) tc::tmem_alloc(&sy.tmem, C::kCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = sy.tmem;
    const int tiles = a.tiles_m * a.tiles_n, first = blockIdx.x, stride = gridDim.x;
    const int idle = PROBE ? a.idle : -1;

    if (warp == kProducer && lane == 0 && idle != kRoleProducer) {
        // producer: the blocks of every k-stage of every tile of this CTA
        // operands that other tiles read too stay in L2 against the stream of results; weights
        // for one row of tiles are read once
        uint64_t keep, weights;
        asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        weights = a.tiles_m > 1 ? keep : policy_evict_first();
        const int blocks_n = blocks_of(a.N, kRows);
        // (this thread is on the way of every stage's refill: pointers and phases run along)
        const size_t next_block = static_cast<size_t>(a.nk) * kBlock;
        uint32_t it = 0, s = 0, phase = 1;   // the phase of `empty` before the current use of the slot
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += stride) {
            const int tm = tile % a.tiles_m, tn = tile / a.tiles_m, nb = min(C::kNB, blocks_n - tn * C::kNB);
            const uint32_t bytes = static_cast<uint32_t>(kBlock * (1 + nb));
            const uint8_t* src_a = a.a + static_cast<size_t>(tm) * next_block;
            const uint8_t* src_b = a.b + static_cast<size_t>(tn * C::kNB) * next_block;
            const uint8_t* src_c = src_b + next_block;   // the second weight block
            for (int k = 0; k < a.nk; ++k, ++it, src_a += kBlock, src_b += kBlock, src_c += kBlock) {
                if (it >= static_cast<uint32_t>(kStages) && !(ok = wait_or_abort<PROBE>(sy, &sy.empty[s], phase, a))) break;
                uint8_t* st = smem + s * C::kStageBytes;
                mbar_arrive_expect_tx(&sy.full[s], bytes);
                bulk_g2s(st, src_a, kBlock, &sy.full[s], keep);
                // codes of the weight blocks side by side, then their scales
                bulk_g2s(st + C::kB, src_b, kCodes, &sy.full[s], weights);
                if (nb > 1) bulk_g2s(st + C::kB + kCodes, src_c, kCodes, &sy.full[s], weights);
                bulk_g2s(st + C::kSf, src_b + kCodes, kScales, &sy.full[s], weights);
                if (nb > 1) bulk_g2s(st + C::kSf + kScales, src_c + kCodes, kScales, &sy.full[s], weights);
                if (++s == static_cast<uint32_t>(kStages)) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // the copies in flight land before the CTA ends, whoever gave up (bounded)
        for (uint32_t b = it > static_cast<uint32_t>(kStages) ? it - kStages : 0; b < it; ++b)
            mbar_wait(&sy.full[b % kStages], (b / kStages) & 1, kDrainRounds);
        if (PROBE) sy.copies = it;
    } else if (warp == kIssuer && lane == 0 && idle != kRoleIssuer) {
        // issuer
        constexpr uint32_t kIdesc = tc::idesc_nvf4(kRows, TN);
        uint32_t it = 0, n = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += stride, ++n) {
            const uint32_t buf = n % C::kAcc, use = n / C::kAcc;
            if (use > 0 && !(ok = wait_or_abort<PROBE>(sy, &sy.acc_empty[buf], (use - 1) & 1, a))) break;
            for (int k = 0; k < a.nk; ++k, ++it) {
                const uint32_t s = it % kStages;
                // the scales are stored, hence the operands have landed
                if (!(ok = wait_or_abort<PROBE>(sy, &sy.sf_full[s], (it / kStages) & 1, a))) break;
                tc::fence_after_sync();
                const uint32_t st = smem_u32(smem + s * C::kStageBytes);
                const uint64_t da = tc::desc_operand(st), db = tc::desc_operand(st + C::kB);
                const uint32_t sfa = tmem + C::kSfA + s * C::kSfStep, sfb = tmem + C::kSfB + s * C::kSfStep;
#pragma unroll
                for (int j = 0; j < 4; ++j)   // 64 of k: 32 bytes of the 128-byte rows
                    tc::mma_nvf4(tmem + buf * TN, da + 2 * j, db + 2 * j, kIdesc, sfa + 4 * j, sfb + 4 * C::kNB * j, k > 0 || j > 0);
                tc::commit(&sy.empty[s]);
            }
            if (ok) tc::commit(&sy.acc_full[buf]);
        }
        // the issued instructions finish before tensor memory is freed, whoever gave up (bounded;
        // a barrier of their own: an accumulator's phases depend on where this loop was left)
        tc::commit(&sy.issued);
        mbar_wait(&sy.issued, 0, kDrainRounds);
    } else if (warp >= kEpiWarps && warp < kProducer && idle != kRoleScales) {
        // scales: shared memory -> registers -> this warp's 32 lanes of tensor memory
        const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t group = static_cast<uint32_t>(warp - kEpiWarps) / kSfWarps;
        uint32_t it = 0;
        bool ok = true;
        for (int tile = first; ok && tile < tiles; tile += stride) {
            for (int k = 0; k < a.nk; ++k, ++it) {
                if (it % kSfGroups != group) continue;
                const uint32_t s = it % kStages;
                // (a landed stage means that its slot's last one, and so its scales, have been multiplied)
                ok = __all_sync(0xFFFFFFFFu, wait_or_abort<PROBE>(sy, &sy.full[s], (it / kStages) & 1, a));
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t st = smem_u32(smem + s * C::kStageBytes) + lane * 16;
                uint32_t w[C::kSfStep];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    lds16(st + kCodes + 512 * j, w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
#pragma unroll
                    for (int b = 0; b < C::kNB; ++b) {
                        const int o = 16 + 4 * (C::kNB * j + b);
                        lds16(st + C::kSf + b * kScales + 512 * j, w[o], w[o + 1], w[o + 2], w[o + 3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < C::kSfStep; j += 16) tc::tmem_store16(at + C::kSfA + s * C::kSfStep + j, w + j);
                tc::tmem_store_wait();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sy.sf_full[s]);
            }
        }
    } else if (warp < kEpiWarps && idle != kRoleEpilogue) {
        const float gb = __ldg(a.gb);
        const int quarter = warp & 3, part = warp >> 2;
        const bool vec = (reinterpret_cast<uintptr_t>(a.y) & 31u) == 0 && (a.ldy * static_cast<long long>(sizeof(TY))) % 32 == 0;
        uint32_t n = 0;
        for (int tile = first; tile < tiles; tile += stride, ++n) {
            const int m = (tile % a.tiles_m) * kRows + quarter * 32 + lane, n0 = (tile / a.tiles_m) * TN + part * kCols;
            const float g = m < a.M ? a.ga[m] * gb : 0.0f;
            const uint32_t buf = n % C::kAcc, acc = tmem + (static_cast<uint32_t>(quarter) << 21) + buf * TN + part * kCols;
            const bool ok = wait_or_abort<PROBE>(sy, &sy.acc_full[buf], (n / C::kAcc) & 1, a);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            tc::fence_after_sync();
            TY* row = static_cast<TY*>(a.y) + static_cast<size_t>(m) * a.ldy + n0;
            if constexpr (sizeof(TY) == 2) {
                constexpr int kChunks = kCols / 16, kHeld = kChunks < 2 ? kChunks : 2;
                const auto read = [&](int c, uint32_t* w) {   // 16 results, rounded
                    uint32_t r[16];
                    tc::tmem_load16(acc + 16 * c, r);
                    tc::tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = rows::Elem<TY>::pack2(__uint_as_float(r[2 * i]) * g, __uint_as_float(r[2 * i + 1]) * g);
                };
                const auto write = [&](int c, const uint32_t* w) {
                    if (m >= a.M || n0 + 16 * c >= a.N) return;
                    if (vec) {
                        store32(row + 16 * c, w);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            reinterpret_cast<uint16_t*>(row)[16 * c + 2 * i] = static_cast<uint16_t>(w[i]);
                            reinterpret_cast<uint16_t*>(row)[16 * c + 2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
                        }
                    }
                };
                // the last two chunks are stored after the accumulators are free (all four held
                // spill registers: 586 us against 567)
#pragma unroll
                for (int c = 0; c < kChunks - kHeld; ++c) {
                    uint32_t w[8];
                    read(c, w);
                    write(c, w);
                    __syncwarp();
                }
                uint32_t w[kHeld][8];
#pragma unroll
                for (int c = 0; c < kHeld; ++c) read(kChunks - kHeld + c, w[c]);
                tc::fence_before_sync();
                if (lane == 0) mbar_arrive(&sy.acc_empty[buf]);
#pragma unroll
                for (int c = 0; c < kHeld; ++c) write(kChunks - kHeld + c, w[c]);
            } else {   // this many 32-bit results do not fit beside the rest: store as they are read
                for (int c = 0; c < kCols / 16; ++c) {
                    uint32_t r[16];
                    tc::tmem_load16(acc + 16 * c, r);
                    tc::tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * g);
                    if (m < a.M && n0 + 16 * c < a.N) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if (vec) {
                                store32(row + 16 * c + 8 * i, &r[8 * i]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; ++j) row[16 * c + 8 * i + j] = __uint_as_float(r[8 * i + j]);
                            }
                        }
                    }
                    __syncwarp();
                }
                tc::fence_before_sync();
                if (lane == 0) mbar_arrive(&sy.acc_empty[buf]);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (PROBE && threadIdx.x == 0) {
        bool done = idle == kRoleIssuer || mbar_test(&sy.issued, 0);
        for (uint32_t i = 0; i < static_cast<uint32_t>(kStages); ++i)   // the last use of slot i
            if (i < sy.copies) done = mbar_test(&sy.full[i], ((sy.copies - 1 - i) / kStages) & 1) && done;
        if (!done && a.error != nullptr) atomicOr(a.error, kDevErrUnfinished);
    }
    if (warp == 0) tc::tmem_free(tmem, C::kCols);
}

template <class TY, int TN, bool PROBE>
static cudaError_t launch_product(Args a, cudaStream_t s) {
    using C = Cfg<TN>;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    a.tiles_n = blocks_of(a.N, TN);
    const long long tiles = static_cast<long long>(a.tiles_m) * a.tiles_n;
    constexpr int kDevices = 64;
    static std::atomic<bool> known[kDevices];   // per device: the kernel's shared memory has been allowed
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(product_kernel<TY, TN, PROBE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        known[dev].store(true, std::memory_order_release);
    }
    product_kernel<TY, TN, PROBE><<<static_cast<unsigned>(tiles < sms ? tiles : sms), kThreads, C::kSmem, s>>>(a);
    return cudaGetLastError();
}

template <class T>
static cudaError_t launch_quantize(const void* x, long long ldx, int M, int K, uint8_t* out, float* scale, cudaStream_t s) {
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (M == 1 || (ldx * static_cast<long long>(sizeof(T))) % 16 == 0);
    if (vec) quantize_kernel<T, true><<<M, kQThreads, 0, s>>>(static_cast<const T*>(x), ldx, K, out, scale);
    else quantize_kernel<T, false><<<M, kQThreads, 0, s>>>(static_cast<const T*>(x), ldx, K, out, scale);
    return cudaGetLastError();
}

template <class TY, bool PROBE = false>
static cudaError_t launch_tiles(const Args& a, cudaStream_t s) {
    // Wide tiles read fewer operand bytes per product, narrow ones spread a small
    // product over more SMs. By rounds of tiles times the tile's width, wide where that
    // is at most an eighth more (us, wide / narrow): 8,192 x 64,064 x 2,560 602 / 745,
    // 517 x 4,608 x 2,560 11.6 / 13.4 (one round against two), 32 x 2,560 x 5,120
    // 14.8 / 13.3, 100 x 64,064 x 2,560 26.7 / 27.0 (before the last two steps above).
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const auto cost = [&](int tn) {
        const long long tiles = static_cast<long long>(a.tiles_m) * blocks_of(a.N, tn);
        return (tiles + sms - 1) / sms * tn;
    };
    return 8 * cost(256) <= 9 * cost(128) ? launch_product<TY, 256, PROBE>(a, s) : launch_product<TY, 128, PROBE>(a, s);
}

}  // namespace mm

size_t matmul_packed_bytes(int N, int K) {
    return static_cast<size_t>(mm::blocks_of(N, mm::kRows)) * mm::blocks_of(K, mm::kStageK) * mm::kBlock;
}

size_t matmul_workspace_bytes(int M, int K) {
    return matmul_packed_bytes(M, K) + (static_cast<size_t>(M) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_matmul_pack(const uint8_t* q, const uint8_t* sf, int N, int K, uint8_t* out, cudaStream_t s) {
    const size_t total = matmul_packed_bytes(N, K) / mm::kBlock * mm::kRows * 8;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const size_t want = (total + 255) / 256, cap = static_cast<size_t>(sms) * 8;
    mm::pack_kernel<<<static_cast<unsigned>(want < cap ? want : cap), 256, 0, s>>>(q, sf, N, K, out);
    return cudaGetLastError();
}

cudaError_t launch_matmul(const MatmulArgs& m, cudaStream_t s) {
    uint8_t* blocks = static_cast<uint8_t*>(m.ws);
    float* scale = reinterpret_cast<float*>(blocks + matmul_packed_bytes(m.M, m.K));
    cudaError_t e = m.x_type == DH_T_BF16  ? mm::launch_quantize<__nv_bfloat16>(m.x, m.ldx, m.M, m.K, blocks, scale, s)
                    : m.x_type == DH_T_F16 ? mm::launch_quantize<__half>(m.x, m.ldx, m.M, m.K, blocks, scale, s)
                                           : mm::launch_quantize<float>(m.x, m.ldx, m.M, m.K, blocks, scale, s);
    if (e != cudaSuccess) return e;
    mm::Args a = {};
    a.a = blocks;
    a.b = m.packed;
    a.ga = scale;
    a.gb = m.g;
    a.y = m.y;
    a.ldy = m.ldy;
    a.M = m.M;
    a.N = m.N;
    a.nk = mm::blocks_of(m.K, mm::kStageK);
    a.tiles_m = mm::blocks_of(m.M, mm::kRows);
    a.error = m.error;
    if (m.probe_rounds != 0) {
        a.idle = m.probe_role;
        a.rounds = m.probe_rounds;
        return mm::launch_tiles<__nv_bfloat16, true>(a, s);
    }
    switch (m.y_type) {
        case DH_T_BF16: return mm::launch_tiles<__nv_bfloat16>(a, s);
        case DH_T_F16: return mm::launch_tiles<__half>(a, s);
        default: return mm::launch_tiles<float>(a, s);
    }
}

}  // namespace dh
