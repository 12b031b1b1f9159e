// Softmax cross entropy of hidden states against a vocabulary given by its head rows, and
// its gradients, without the T x N logits in memory (g, below, is: in 16 bits, a piece of the
// vocabulary at a time).
//
//   z_tn = h_t . W_n,  m_t = max_n z_tn,  S_t = sum_n e^(z_tn - m_t),
//   lse_t = m_t + ln S_t,  loss_t = w_t (ln S_t + (m_t - z_ty)),
//   g_tn = w_t (e^(z_tn - lse_t) - [n = y_t]),  dh = g W,  dW = g^T h.
//
// Loss: one product (dh_gemm.cuh) whose epilogue keeps, per token and 128 columns, the running
// maximum and sum; 8 bytes for every 128 logits are written and joined by a second kernel.
// Gradients: the vocabulary is taken in pieces; the piece's logits are multiplied again, its g
// is written in 16 bits (the only [tokens x piece] array), and two products read it, one along
// the piece (dh, added up over the pieces in 32 bits), one along the tokens (dW, final). The
// product is three quarters useful: 8 T N K operations against the 6 that the mathematics has,
// the price of keeping no logits between the loss and the gradients. (For up to 128 tokens the
// logits, T x N of them, are less than the piece may take anyway, and reading the head again would be
// the work: a call that computes both keeps them in its workspace between its products.)
//
// Roundings besides 32-bit arithmetic: g to the inputs' 16-bit type (the tensor cores take
// nothing wider from it; its error is that of rounding the results again), scaled by a power of
// two so that the largest row weight lies just under 1 (bf16) or 2^15 (f16, whose probabilities
// would be subnormal below 6e-5), in two terms for few tokens, small products, or where the caller
// asks for them; the gradients once, at the end.
//
// What bounds it. Many tokens: the tensor cores, whose pipe is busy for 95 to 97 of 100 cycles in
// all four products, at the clock that the power limit leaves them (1.6 of 2.07 GHz): the loss of
// 4,095 x 64,026 x 2,560 takes 690 us (1,950 TFLOP/s), the step of 4,096 2,930 (1,830 over its 8 TNK).
// Few tokens: reading the head, 61 x 64,026 in 60 us (5.5 TB/s), and for a small vocabulary the
// chain of launches, 16 x 4,000 in 21 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dh_gemm.cuh"
#include "dh_rows.cuh"

namespace dh {
namespace ce {

using gemm::Acc;
using gemm::ceil_div;
using gemm::Tile;
using rows::kLog2e;
using rows::kNegInf;

constexpr int kTM = 256, kTN = 256, kPair = 2;
constexpr int kHalf = kTN / 2;   // columns of an epilogue warp

__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Tokens {
    const int32_t* ids;      // [T]
    const int32_t* row_of;   // [V] or null
    const float* weight;     // [T] or null (1)
    int V, T, N;
    // Head row of token t, -1 where it has none.
    __device__ __forceinline__ int row(int t) const {
        int id = ids[t];
        if (row_of != nullptr) id = id >= 0 && id < V ? row_of[id] : -1;
        return id >= 0 && id < N ? id : -1;
    }
    __device__ __forceinline__ float w(int t) const { return weight != nullptr ? weight[t] : 1.0f; }
    // Whether token t counts.
    __device__ __forceinline__ bool live(int t) const { return w(t) != 0.0f && row(t) >= 0; }
};

// The power of two by which row weights are scaled before g is rounded: the largest finite
// one's exponent (bits of |w|) is brought to -1, or to 14 for f16.
template <bool F16>
__device__ __forceinline__ int scale_exponent(uint32_t wmax) {
    const int e = static_cast<int>(wmax >> 23) - 127;   // floor(log2); -127 for subnormals and 0
    return (F16 ? 14 : -1) - (e < -100 ? -100 : e > 126 ? 126 : e);
}

// ---------------------------------------------------------------- the loss ----

// The tensor cores' 32-bit sums are truncated, not rounded, as they grow: over the 160
// instructions of 2,560 features a large logit loses 2e-6 of itself, four times what a product
// in 32 bits is off by. So they sum some steps of 64 features at a time, which the epilogue adds
// up, rounded: the loss of 4,095 x 64,026 was off by 1.8e-6, and is by 3.4e-7 with eight steps, as a
// sum in 32 bits is. That of fewer features is off by less: there four steps (lse of 385 x 595 x 416
// off by 1.3e-7, 2.2e-7 with eight; 4,096 x 64,026 x 416 159 us, 148; x 2,560 776, 743), and two where
// reading the head is the work (24 x 308 x 576 9.1e-8, 1.4e-7 with four, the same time).
int logit_chunk(int P, int steps) { return P == 1 ? 2 : steps <= 16 ? 4 : 8; }

// A thread's 128 columns of one row, its accumulators added up.
template <class L>
__device__ __forceinline__ bool sum_chunks(Acc<L>& acc, int steps, int chunk, uint32_t offset, float (&z)[kHalf]) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i) z[i] = 0.0f;
#pragma unroll 1
    for (int k = 0; k < steps; k += chunk) {
        const uint32_t at = acc.next();
        if (at == ~0u) return false;
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
            uint32_t r[16];
            tc::tmem_load16(at + offset + c, r);
            tc::tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) z[c + i] += __uint_as_float(r[i]);
        }
        acc.release();
    }
    return true;
}

template <class T, int P>
struct Stats {
    using Layout = gemm::Layout<P, kTN, 2, false, false>;
    static constexpr int kFormat = std::is_same<T, __half>::value ? 0 : 1, kChunk = gemm::kPerLaunch;
    static constexpr bool kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        Tokens tok;
        float2* part;   // [2 tiles_n][T]: maximum and sum of 128 columns
        float* target;  // [T]: the token's logit
        uint32_t* wmax; // cleared for what follows
        float* z;       // the logits, [T][ldz] (ldz a multiple of 256), or null
        int ldz;
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * P + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf, valid = a.tok.N - n0;
        const int j = (row < a.tok.T ? a.tok.row(row) : -1) - n0;
        if (row == 0 && n0 == 0) *a.wmax = 0u;
        float z[kHalf];
        if (!sum_chunks(acc, t.steps, a.shape.chunk, (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf, z)) return false;
        if (valid < kHalf) {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) z[i] = i < valid ? z[i] : kNegInf;
        }
        if (P == 1 && a.z != nullptr && row < a.tok.T) {   // (few tokens: single CTAs)
            float* out = a.z + static_cast<size_t>(row) * a.ldz + n0;
#pragma unroll
            for (int i = 0; i < kHalf; i += 8) store32(out + i, reinterpret_cast<const uint32_t*>(&z[i]));
        }
        __syncwarp();
        if (__any_sync(0xFFFFFFFFu, j >= 0 && j < kHalf)) {
            float y = 0.0f;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) y = i == j ? z[i] : y;
            if (j >= 0 && j < kHalf) a.target[row] = y;
            __syncwarp();
        }
        float top[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
        for (int i = 4; i < kHalf; ++i) top[i & 3] = fmaxf(top[i & 3], z[i]);
        const float m = fmaxf(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), kNegInf), ref = m == kNegInf ? 0.0f : m;
        float sum[4] = {};
#pragma unroll
        for (int i = 0; i < kHalf; ++i) sum[i & 3] += exp2_approx((z[i] - ref) * kLog2e);
        if (row < a.tok.T) a.part[static_cast<size_t>(2 * t.n + half) * a.tok.T + row] = make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
        return true;
    }
};

// What the gradients need of a row: the largest finite row weight in use (bits of its
// magnitude), and, where dW is wanted, the hidden states with zeros in the rows that are left
// out: their g is 0, but 0 times what a padding row may hold (infinities, NaN) is not.
struct Rows {
    const void* hidden;      // 16-bit rows
    long long ld;
    int K;
    void* copy;              // [T][K] or null
    int again;               // rows further on, the copy's second one (0: none)
    uint32_t* wmax;
    __device__ __forceinline__ void weigh(float w, bool live) const {
        const uint32_t bits = __float_as_uint(w) & 0x7FFFFFFFu;
        if (live && bits < 0x7F800000u) atomicMax(wmax, bits);   // (a maximum: the order does not matter)
    }
    __device__ __forceinline__ void move(int t, bool live, int i, int step) const {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(hidden) + static_cast<size_t>(t) * ld);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(copy) + static_cast<size_t>(t) * K);
        const size_t second = static_cast<size_t>(again) * (K / 8);
        for (; i < K / 8; i += step) {
            const uint4 v = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
            dst[i] = v;
            if (second != 0) dst[second + i] = v;
        }
    }
};

// Joins the parts: 8 tokens per CTA, the CTA's 1,024 threads over the parts, then over the
// threads of a token. With gradients to come it prepares their rows too.
constexpr int kJoinTokens = 8, kJoinThreads = 1024, kJoinWarps = kJoinThreads / 32;
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2), ref = top == kNegInf ? 0.0f : top;
    s = s * exp2_approx((m - ref) * kLog2e) + s2 * exp2_approx((m2 - ref) * kLog2e);
    m = top;
}
// A row's normaliser from its maximum and sum: m + ln s, and what rounding that took away. (A
// maximum of -inf is that of no finite logits, as of a hidden state with an infinity: NaN.)
struct Normaliser {
    float m, ln, lse, rest;
    __device__ __forceinline__ Normaliser(float m_, float s) : m(m_), ln(logf(m_ > kNegInf ? s : m_)), lse(m + ln) {
        const float b = lse - m;   // (two-sum)
        rest = (m - (lse - b)) + (ln - b);
    }
    __device__ __forceinline__ float loss(float target) const { return ln + (m - target); }
};
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Tokens tok, const float2* part, int parts, const float* target,
                                                            float* loss, float* lse, float* rest, const Rows rows) {
    programmatic_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, token = threadIdx.x % kJoinTokens, t = blockIdx.x * kJoinTokens + token;
    float m = kNegInf, s = 0.0f;
    if (t < tok.T) {
#pragma unroll 4
        for (int j = threadIdx.x / kJoinTokens; j < parts; j += kJoinThreads / kJoinTokens) {
            const float2 p = part[static_cast<size_t>(j) * tok.T + t];
            join(m, s, p.x, p.y);
        }
    }
#pragma unroll
    for (int o = kJoinTokens; o < 32; o <<= 1) join(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
    __shared__ float2 all[kJoinWarps][kJoinTokens];
    if (lane < kJoinTokens) all[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp == 0 && lane < kJoinTokens && t < tok.T) {
#pragma unroll 4
        for (int j = 1; j < kJoinWarps; ++j) join(m, s, all[j][lane].x, all[j][lane].y);
        const Normaliser n(m, s);
        const float w = tok.w(t);
        const bool live = tok.live(t);
        if (loss != nullptr) loss[t] = live ? w * n.loss(target[t]) : 0.0f;
        if (lse != nullptr) lse[t] = n.lse;
        if (rest != nullptr) rest[t] = n.rest;
        if (rows.wmax != nullptr) rows.weigh(w, live);
    }
    if (rows.copy != nullptr) {
        constexpr int kPer = kJoinThreads / kJoinTokens;   // threads of a row
        const int row = blockIdx.x * kJoinTokens + threadIdx.x / kPer;
        if (row < tok.T) rows.move(row, tok.live(row), threadIdx.x % kPer, kPer);
    }
}

// --------------------------------------------------------------- gradients ----

// The rows' work where there is no loss to join.
__global__ void __launch_bounds__(128) rows_kernel(const Tokens tok, const Rows rows) {
    programmatic_wait();
    const int t = blockIdx.x;
    const float w = tok.w(t);
    const bool live = w != 0.0f && tok.row(t) >= 0;
    if (threadIdx.x == 0) rows.weigh(w, live);
    if (rows.copy != nullptr) rows.move(t, live, threadIdx.x, blockDim.x);
}

// A logit's probability.
__device__ __forceinline__ float probability(float z, float lse, float rest) { return exp2_approx(((z - lse) - rest) * kLog2e); }

// 16 elements of g from the probabilities p of columns c .. c + 15 (the token's own is j), weighted
// by w: rounded to `out`, and what that leaves over to `low` (null: nowhere).
template <class T>
__device__ __forceinline__ void store_weights(float (&p)[16], int j, float w, bool live, T* out, T* low) {
    if (j >= 0 && j < 16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = i == j ? p[i] - 1.0f : p[i];
    }
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] *= w;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = live ? rows::Elem<T>::pack2(p[2 * i], p[2 * i + 1]) : 0u;
    store32(out, v);
    if (low == nullptr) return;
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
        float high[8];
        rows::Elem<T>::unpack(make_uint4(v[i / 2], v[i / 2 + 1], v[i / 2 + 2], v[i / 2 + 3]), high);
#pragma unroll
        for (int k = 0; k < 8; ++k) p[i + k] -= high[k];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = live ? rows::Elem<T>::pack2(p[2 * i], p[2 * i + 1]) : 0u;
    store32(low, v);
}

template <class T, int P>
struct Weights {   // g of a piece
    using Layout = gemm::Layout<P, kTN, 2, false, false>;
    static constexpr bool kF16 = std::is_same<T, __half>::value;
    static constexpr int kFormat = kF16 ? 0 : 1;
    static constexpr int kChunk = gemm::kPerLaunch;
    static constexpr bool kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        Tokens tok;
        const float* lse;
        const float* rest;      // or null
        const uint32_t* wmax;
        T* g;                   // [T][ldg], ldg a multiple of 256
        T* low;                 // what rounding g left over, or null
        int ldg;
        int first, count;       // the piece's rows of the head
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * P + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int c0 = t.n * kTN + half * kHalf;   // in the piece
        int y = -1;
        float w = 0.0f, lse = 0.0f, rest = 0.0f;
        if (row < a.tok.T) {
            y = a.tok.row(row);
            w = y >= 0 ? a.tok.w(row) : 0.0f;
            lse = a.lse[row];
            if (a.rest != nullptr) rest = a.rest[row];
        }
        const bool live = w != 0.0f;
        w = ldexpf(w, scale_exponent<kF16>(*a.wmax));
        float z[kHalf];
        if (!sum_chunks(acc, t.steps, a.shape.chunk, (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf, z)) return false;
        const int j = y - (a.first + c0);
        T* out = a.g + static_cast<size_t>(row) * a.ldg + c0;
        T* low = a.low != nullptr ? a.low + static_cast<size_t>(row) * a.ldg + c0 : nullptr;
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
            float p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = probability(z[c + i], lse, rest);
            if (row < a.tok.T && c0 + c < a.count) store_weights<T>(p, j - c, w, live, out + c, low != nullptr ? low + c : nullptr);
        }
        __syncwarp();
        return true;
    }
};

// g of few tokens from their kept logits, with the join: each CTA joins one token's parts (in the
// order of join_kernel) and takes 4,096 columns.
constexpr int kFewThreads = 256, kFewColumns = kFewThreads * 16;
template <class T>
__global__ void __launch_bounds__(kFewThreads) few_kernel(const Tokens tok, const float* z, int ldz, const float2* part, int parts,
                                                          const float* target, float* loss, float* lse, float* rest, const Rows rows,
                                                          T* g, T* low, int ldg) {
    programmatic_wait();
    constexpr int kSlots = kJoinThreads / kJoinTokens;
    const int t = blockIdx.y, lane = threadIdx.x & 31;
    __shared__ float2 all[kSlots / 4];
    __shared__ uint32_t heaviest[kFewThreads / 32];
    __shared__ float norm[2];
    if (threadIdx.x < kSlots) {
        float m = kNegInf, s = 0.0f;
        for (int j = threadIdx.x; j < parts; j += kSlots) {
            const float2 p = part[static_cast<size_t>(j) * tok.T + t];
            join(m, s, p.x, p.y);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) join(m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
        if ((threadIdx.x & 3) == 0) all[threadIdx.x >> 2] = make_float2(m, s);
    }
    // the largest finite row weight in use
    uint32_t heavy = 0u;
    for (int i = threadIdx.x; i < tok.T; i += kFewThreads) {
        const uint32_t bits = tok.live(i) ? __float_as_uint(tok.w(i)) & 0x7FFFFFFFu : 0u;
        if (bits < 0x7F800000u && bits > heavy) heavy = bits;
    }
    heavy = __reduce_max_sync(~0u, heavy);
    if (lane == 0) heaviest[threadIdx.x >> 5] = heavy;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewThreads / 32; ++i) heavy = max(heavy, heaviest[i]);
    float w = tok.w(t);
    const int y = tok.row(t);
    const bool live = w != 0.0f && y >= 0;
    if (threadIdx.x == 0) {
        float m = all[0].x, s = all[0].y;
        const int groups = (parts < kSlots ? parts + 3 : kSlots) / 4;   // (joining nothing changes nothing)
        for (int j = 1; j < groups; ++j) join(m, s, all[j].x, all[j].y);
        const Normaliser n(m, s);
        norm[0] = n.lse, norm[1] = n.rest;
        if (blockIdx.x == 0) {
            loss[t] = live ? w * n.loss(target[t]) : 0.0f;
            if (lse != nullptr) lse[t] = n.lse;
            if (rest != nullptr) rest[t] = n.rest;
            if (t == 0) *rows.wmax = heavy;
        }
    }
    __syncthreads();
    if (rows.copy != nullptr) rows.move(t, live, static_cast<int>(blockIdx.x) * kFewThreads + threadIdx.x, static_cast<int>(gridDim.x) * kFewThreads);
    const int c = static_cast<int>(blockIdx.x) * kFewColumns + threadIdx.x * 16;
    if (c >= ldg) return;   // (columns beyond N lie outside the products' maps)
    w = ldexpf(w, scale_exponent<std::is_same<T, __half>::value>(heavy));
    float p[16];
    const float4* src = reinterpret_cast<const float4*>(z + static_cast<size_t>(t) * ldz + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 q = __ldcs(src + i);
        p[4 * i] = q.x, p[4 * i + 1] = q.y, p[4 * i + 2] = q.z, p[4 * i + 3] = q.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = probability(p[i], norm[0], norm[1]);
    const size_t at = static_cast<size_t>(t) * ldg + c;
    store_weights<T>(p, y - c, w, live, g + at, low + at);
}

// The gradients' sums are truncated as the logits' are, and their contractions are longer: summed
// throughout by the tensor cores, dW of 1,100,000 tokens was short by 3.7e-4 of itself. Sixteen steps at a
// time leave 4e-6 and cost nothing (4,096 x 64,026 x 2,560 3,076 us, 3,096; 100 x 64,026 236, 233).
constexpr int kGradientChunk = 16;

// A thread's columns of one row (`columns` of 128, a multiple of 8), sixteen at a time to
// put(column, values).
template <class L, class Put>
__device__ __forceinline__ bool each_sixteen(Acc<L>& acc, int steps, uint32_t offset, int columns, Put put) {
    float z[kHalf];
    if (!sum_chunks(acc, steps, kGradientChunk, offset, z)) return false;
#pragma unroll
    for (int c = 0; c < kHalf; c += 16)
        if (c < columns) put(c, z + c);
    __syncwarp();
    return true;
}

// 16 columns (`columns` of them there, 8 or more), scaled and rounded, to `out`: in 32-byte pieces
// where rows are so aligned (`wide`; then all 16 are there), else 16. A row that does not count is
// zeros whatever it was multiplied by.
template <class T>
__device__ __forceinline__ void store_rounded(const float* z, T* out, int columns, float scale, bool live, bool wide) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = live ? rows::Elem<T>::pack2(z[2 * j] * scale, z[2 * j + 1] * scale) : 0u;
    if (wide) {
        store32(out, v);
    } else {
        __stcg(reinterpret_cast<uint4*>(out), make_uint4(v[0], v[1], v[2], v[3]));
        if (columns > 8) __stcg(reinterpret_cast<uint4*>(out + 8), make_uint4(v[4], v[5], v[6], v[7]));
    }
}

// The same as 32-bit sums (rows 32-byte aligned), added to what is there if `add`.
__device__ __forceinline__ void store_sums(const float* z, float* out, int columns, bool add) {
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
        if (i >= columns) break;
        float v[8] = {};
        if (add) {
            const float4 p = *reinterpret_cast<const float4*>(out + i), q = *reinterpret_cast<const float4*>(out + i + 4);
            v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += z[i + j];
        store32(out + i, reinterpret_cast<const uint32_t*>(v));
    }
}

// dh: g (along the piece) times the piece's head rows, as 32-bit sums: [T][K] of whole tiles
// and first parts, then the other parts of the tiles that are split, [split - 1][tile][256][256].
template <class T>
struct Hidden {
    using Layout = gemm::Layout<kPair, kTN, 2, false, true>;
    static constexpr int kFormat = std::is_same<T, __half>::value ? 0 : 1;
    static constexpr int kChunk = kGradientChunk;
    static constexpr bool kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        int T_, K;
        float* sum;
        float* parts;
        int add;      // to what earlier pieces left
        // the results themselves, where one sum is all there is (null: sums)
        T* out;
        long long ld;
        const uint32_t* wmax;
        Tokens tok;
    };
    template <class A2>
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, A2& acc) {
        const int local = rank * gemm::kRows + (warp & 3) * 32 + lane, row = t.m * kTM + local, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf;
        const bool in = row < a.T_;
        const uint32_t offset = (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        const bool live = a.out != nullptr && in && a.tok.live(row);
        const float scale = live ? exp2i(-scale_exponent<std::is_same<T, __half>::value>(*a.wmax)) : 0.0f;
        T* out = a.out + static_cast<size_t>(row) * a.ld + n0;
        float* sums;
        if (t.split <= 0) {
            sums = a.sum + static_cast<size_t>(row) * a.K + n0;
        } else {
            const int rest = a.shape.tiles() - a.shape.whole, at = gemm::tile_index(a.shape.tiles_m, a.shape.tiles_n, t.m, t.n) - a.shape.whole;
            sums = a.parts + (static_cast<size_t>((t.split - 1) * rest + at) * kTM + local) * kTN + half * kHalf;
        }
        return each_sixteen(acc, t.steps, offset, a.K - n0, [&](int c, const float* z) {
            if (!in) return;
            if (a.out != nullptr) store_rounded<T>(z, out + c, a.K - n0 - c, scale, live, false);
            else store_sums(z, sums + c, a.K - n0 - c, a.add != 0);
        });
    }
};

// dW: the piece's g (along the tokens) times the hidden states, final. (Rows stored in 32-byte
// pieces where they are so aligned: backward of 333 x 248,320 1,424 us with 16-byte ones, 1,154.)
template <class T>
struct Head {
    using Layout = gemm::Layout<kPair, kTN, 2, true, true>;
    static constexpr bool kF16 = std::is_same<T, __half>::value;
    static constexpr int kFormat = kF16 ? 0 : 1;
    static constexpr int kChunk = kGradientChunk;
    static constexpr bool kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        int rows, K;             // head rows of the piece
        const uint32_t* wmax;
        T* out;                  // the piece's first row
        long long ld;
        int wide;                // rows 32-byte aligned
        float* parts;            // the tokens in parts: their sums, [split][tile][256][256] (null: results)
    };
    template <class A2>
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, A2& acc) {
        const int row = (t.m * kPair + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf;
        const bool in = row < a.rows;
        const uint32_t offset = (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        const int at = gemm::tile_index(a.shape.tiles_m, a.shape.tiles_n, t.m, t.n);
        float* sums = a.parts + ((static_cast<size_t>(t.split) * a.shape.tiles() + at) * kTM + rank * gemm::kRows + (warp & 3) * 32 + lane) * kTN +
                      half * kHalf;
        const float scale = exp2i(-scale_exponent<kF16>(*a.wmax));
        T* out = a.out + static_cast<size_t>(row) * a.ld + n0;
        return each_sixteen(acc, t.steps, offset, a.K - n0, [&](int c, const float* z) {
            if (!in) return;
            if (a.parts != nullptr) store_sums(z, sums + c, a.K - n0 - c, false);
            else store_rounded<T>(z, out + c, a.K - n0 - c, scale, true, a.wide);
        });
    }
};

// dh from its sums, and dW from those of its parts: eight elements per thread, parts in order.
// Rows of dh that are left out are zeros whatever the head holds.
struct Sums {
    size_t elements;           // of dh, in eights (0: none)
    const float* sum;
    const float* parts;
    int tiles_m, tiles_n, whole, splits, terms;
    void* out;
    long long ld;
    // dW
    gemm::Shape head;          // its tiles, all in parts (splits; none: 0)
    const float* head_parts;
    void* head_out;
    long long head_ld;
    int head_rows;
};
__device__ __forceinline__ void add8(float (&v)[8], const float* p) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
    v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w, v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
}
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(const Tokens tok, const Sums a, int K, const uint32_t* wmax) {
    programmatic_wait();
    const float scale = exp2i(-scale_exponent<std::is_same<T, __half>::value>(*wmax));
    const unsigned per_row = K / 8;
    constexpr unsigned kTile = kTM * kTN / 8;
    const size_t head = static_cast<size_t>(a.head.tiles()) * kTile;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < a.elements + head; i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        float v[8] = {};
        T* out;
        if (i < a.elements) {
            const int row = static_cast<int>(i / per_row), col = static_cast<int>(i % per_row) * 8;
            out = static_cast<T*>(a.out) + static_cast<size_t>(row) * a.ld + col;
            for (int e = 0; e < a.terms; ++e) {
                const int r = row + e * tok.T;
                add8(v, a.sum + static_cast<size_t>(r) * K + col);
                const int at = gemm::tile_index(a.tiles_m, a.tiles_n, r / kTM, col / kTN) - a.whole;
                if (at < 0) continue;
                const size_t step = static_cast<size_t>(a.tiles_m * a.tiles_n - a.whole) * kTM * kTN;
                const float* p = a.parts + (static_cast<size_t>(at) * kTM + r % kTM) * kTN + col % kTN;
                for (int s = 1; s < a.splits; ++s, p += step) add8(v, p);
            }
            const bool live = tok.live(row);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = live ? v[j] * scale : 0.0f;
        } else {
            const unsigned at = static_cast<unsigned>((i - a.elements) / kTile), in = static_cast<unsigned>((i - a.elements) % kTile) * 8;
            gemm::Shape whole = a.head;
            whole.whole = whole.tiles();
            const Tile t = gemm::tile_at(whole, static_cast<int>(at));
            const int row = t.m * kTM + static_cast<int>(in / kTN), col = t.n * kTN + static_cast<int>(in % kTN);
            if (row >= a.head_rows || col >= K) continue;
            out = static_cast<T*>(a.head_out) + static_cast<size_t>(row) * a.head_ld + col;
            const float* p = a.head_parts + static_cast<size_t>(at) * kTM * kTN + in;
            for (int s = 0; s < a.head.splits; ++s, p += static_cast<size_t>(a.head.tiles()) * kTM * kTN) add8(v, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= scale;
        }
        *reinterpret_cast<uint4*>(out) = rows::Elem<T>::pack(v);
    }
}

// ------------------------------------------------------------------- host ----

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Head rows per piece: g of a piece takes at most 512 MiB (or 2,048 rows where the tokens are
// many).
int piece_rows(int T, int N) {
    const long long fit = (1ll << 28) / T / kTN * kTN, least = fit < 2048 ? 2048 : fit;
    const long long all = static_cast<long long>(ceil_div(N, kTN)) * kTN;
    return static_cast<int>(least < all ? least : all);
}

// dh's tiles: whole ones as long as they fill all pairs of SMs, the rest in parts (at least
// eight steps long) such that its rounds take the fewest steps, a part counted as eight more and
// the sum of parts as twelve.
// 4,096 x 64,026 x 2,560 (160 tiles for 76 pairs, the last 8 in parts): the step 3,591 us with three
// rounds of whole tiles, 2,985.
gemm::Shape hidden_tiles(int T, int K, int piece, unsigned int* error) {
    gemm::Shape s = gemm::whole_tiles(ceil_div(T, kTM), ceil_div(K, kTN), ceil_div(piece, 64), error);
    constexpr int pairs = kSms / kPair;
    const int rest = s.whole % pairs;
    if (rest == 0) return s;
    s.whole -= rest;
    long long least = 0;
    for (int p = 1; p <= 32 && (p == 1 || s.steps / p >= 8); ++p) {
        const long long cost = static_cast<long long>(ceil_div(rest * p, pairs)) * ceil_div(s.steps, p) + (p > 1 ? 12 + 8 * p : 0);
        if (p == 1 || cost < least) {
            least = cost;
            s.split_steps = ceil_div(s.steps, p);
        }
    }
    s.splits = ceil_div(s.steps, s.split_steps);
    return s;
}

// g in two terms, its 16-bit rounding and what that left over, as rows T .. 2 T - 1 of g, of dh's
// sums and (the same hidden states again) of dW's contraction. One term makes the gradients' error
// 1.43 times that of rounding them alone (64,026 x 2,560 bf16, relative 2-norm: 0.00238 and 0.00166), and
// up to 1.6 times where they are sums of few terms (191 x 230 x 128); a second one takes it away at any
// size. So there are two where that costs little: for up to 128 tokens, for which the products' tiles
// have the room, and for small products of up to 1,024, whose time is their launches' (device us, one term
// / two: 200 x 230 x 128 18.6 / 20.7, 129 x 4,000 x 256 27.5 / 29.1, 256 x 4,096 x 256, T N K of 2^28,
// 28.1 / 29.7). Beyond, it is the caller's choice (DH_CE_TWO_TERMS): 2^30 of 1,000 tokens 31.5 / 36.6, of
// 4,096 50 / 61; 64,026 x 2,560, 129 tokens 276 / 336, 520 513 / 705, 4,096 2,776 / 4,482. (The error is
// within the gradients' own type; who keeps 16-bit logits has it as well.)
int terms_of(int T, int N, int K, bool two_terms) {
    return two_terms || T <= 128 || (T <= 1024 && static_cast<long long>(T) * N * K <= 1ll << 28) ? 2 : 1;
}

// dW's tiles where they are few and the tokens many: all in parts of at least eight steps, as many
// as fill the pairs of SMs once (6,208 tokens, 5 rows of 4,592: 34 us of 105 were 18 tiles of 97
// steps). A head of several pieces has tiles enough.
gemm::Shape head_tiles(int rows, int N, int K, int piece, unsigned int* error) {
    gemm::Shape s = gemm::whole_tiles(ceil_div(N, kTM), ceil_div(K, kTN), ceil_div(rows, 64), error);
    constexpr int pairs = kSms / kPair;
    if (N > piece || s.tiles() > pairs / 2 || s.steps < 16) return s;
    const int p = pairs / s.tiles() < s.steps / 8 ? pairs / s.tiles() : s.steps / 8;
    s.whole = 0;
    s.split_steps = ceil_div(s.steps, p);
    s.splits = ceil_div(s.steps, s.split_steps);
    return s;
}

// Whether a call for both keeps its logits: few tokens whose vocabulary is one piece. Multiplied
// again, 12 x 83,361 x 3,568 takes 449 us; kept, 347 (the head is read twice in place of three times).
bool keeps_logits(int T, int N) { return T <= gemm::kRows && N <= piece_rows(2 * T, N); }

struct Space {
    size_t z, wmax, part, target, lse, rest, g, hidden, sum, parts, head_parts, bytes;
};
Space space_of(int T, int N, int K, bool loss, bool dh, bool dw, bool two_terms) {
    Space s = {};
    size_t at = 256;   // wmax at 0
    const auto take = [&](size_t n) {
        const size_t here = at;
        at += up256(n);
        return here;
    };
    const size_t t = static_cast<size_t>(T);
    if (loss) {
        s.part = take(t * 2 * ceil_div(N, kTN) * sizeof(float2));
        s.target = take(t * 4);
        s.lse = take(t * 4);
        s.rest = take(t * 4);
    }
    const int rows = terms_of(T, N, K, two_terms) * T, piece = piece_rows(rows, N);
    const size_t r = static_cast<size_t>(rows);
    if (dh || dw) s.g = take(r * piece * 2);
    if (loss && (dh || dw) && keeps_logits(T, N)) s.z = take(t * up256(N) * 4);
    if (dw) {
        s.hidden = take(r * K * 2);
        const gemm::Shape w = head_tiles(rows, N, K, piece, nullptr);
        if (w.whole == 0) s.head_parts = take(static_cast<size_t>(w.units()) * kTM * kTN * 4);
    }
    if (dh) {
        const gemm::Shape h = hidden_tiles(rows, K, piece, nullptr);
        s.sum = take(r * K * 4);
        s.parts = take(static_cast<size_t>(h.tiles() - h.whole) * (h.splits - 1) * kTM * kTN * 4);
    }
    s.bytes = at;
    return s;
}

// P: CTAs of a tile of the logits. Single ones for up to 128 tokens, which fill no pair's 256 rows
// (their products are bound by reading the head: 61 x 64,026 67 us in pairs, 59), pairs otherwise
// (two thirds of the loads).
template <class T, int P>
cudaError_t run(const CrossEntropyArgs& c, cudaStream_t stream) {
    const bool loss = c.loss != nullptr, dh = c.dhidden != nullptr, dw = c.dhead != nullptr;
    const Space sp = space_of(c.T, c.N, c.K, loss, dh, dw, c.two_terms);
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    Tokens tok = {c.tokens, c.row_of, c.weight, c.V, c.T, c.N};
    uint32_t* wmax = reinterpret_cast<uint32_t*>(ws + sp.wmax);
    const int tiles_m = ceil_div(c.T, gemm::kRows * P);
    T* hidden = dw ? reinterpret_cast<T*>(ws + sp.hidden) : nullptr;
    const int terms = terms_of(c.T, c.N, c.K, c.two_terms), all_rows = terms * c.T;   // of g
    const Rows rows = {c.hidden, c.ld_hidden, c.K, hidden, terms > 1 ? c.T : 0, wmax};
    cudaError_t e;
    using K1 = typename Stats<T, P>::Layout;
    gemm::Jobs<Stats<T, P>> logits = {};
    gemm::Jobs<Weights<T, P>> pieces = {};
    CUtensorMap &map_h = logits.first.map_a, &map_w = logits.first.map_b;
    if ((e = gemm::encode_operand<K1, false>(&map_h, c.hidden, c.T, c.K, c.ld_hidden * 2, gemm::kRows)) != cudaSuccess) return e;
    if ((e = gemm::encode_operand<K1, false>(&map_w, c.head, c.N, c.K, c.ld_head * 2, K1::kBRows)) != cudaSuccess) return e;
    pieces.first.map_a = map_h;
    pieces.first.map_b = map_w;
    const int steps = ceil_div(c.K, K1::kK);
    const bool kept = P == 1 && loss && (dh || dw) && keeps_logits(c.T, c.N);
    const float2* part = reinterpret_cast<const float2*>(ws + sp.part);
    const float* lse = c.lse_in;
    const float* rest = c.rest_in;
    if (loss) {
        typename Stats<T, P>::Args& a = logits.first.args;
        a.shape = gemm::whole_tiles(tiles_m, ceil_div(c.N, kTN), steps, c.error);
        a.shape.chunk = logit_chunk(P, steps);
        a.shape.rounds = c.probe_rounds;
        a.shape.idle = c.probe_role;
        a.tok = tok;
        a.part = reinterpret_cast<float2*>(ws + sp.part);
        a.target = reinterpret_cast<float*>(ws + sp.target);
        a.wmax = wmax;
        if (kept) {
            a.z = reinterpret_cast<float*>(ws + sp.z);
            a.ldz = static_cast<int>(up256(c.N));
        }
        if ((e = gemm::launch(logits, stream)) != cudaSuccess) return e;
        float* l = c.lse != nullptr ? c.lse : reinterpret_cast<float*>(ws + sp.lse);
        float* r = c.rest != nullptr ? c.rest : reinterpret_cast<float*>(ws + sp.rest);
        if (!kept)
            e = gemm::launch_early(join_kernel, dim3(static_cast<unsigned>(ceil_div(c.T, kJoinTokens))), kJoinThreads, 0, 1, stream, tok, a.part,
                                   2 * a.shape.tiles_n, a.target, c.loss, l, r, dh || dw ? rows : Rows{});
        if (e != cudaSuccess) return e;
        lse = l;
        rest = r;
    }
    if (!dh && !dw) return cudaSuccess;

    if (!loss) {
        if ((e = cudaMemsetAsync(wmax, 0, 4, stream)) != cudaSuccess) return e;
        if ((e = gemm::launch_early(rows_kernel, dim3(static_cast<unsigned>(c.T)), 128, 0, 1, stream, tok, rows)) != cudaSuccess) return e;
    }
    const int piece = piece_rows(all_rows, c.N);
    const gemm::Shape tiles_h = hidden_tiles(all_rows, c.K, piece, c.error);   // of a full piece
    const gemm::Shape tiles_w = head_tiles(all_rows, c.N, c.K, piece, c.error);
    float* head_parts = dw && tiles_w.whole == 0 ? reinterpret_cast<float*>(ws + sp.head_parts) : nullptr;
    T* g = reinterpret_cast<T*>(ws + sp.g);
    float* sum = reinterpret_cast<float*>(ws + sp.sum);
    const bool direct = terms == 1 && c.N <= piece && ceil_div(ceil_div(c.N, 64), tiles_h.split_steps) == 1;   // dh is one sum
    int splits = 1;   // of dh's split tiles: those of the first piece, which is the largest
    for (int first = 0; first < c.N; first += piece) {
        const int count = c.N - first < piece ? c.N - first : piece;
        typename Weights<T, P>::Args& a = pieces.first.args;
        a.shape = gemm::whole_tiles(tiles_m, ceil_div(count, kTN), steps, c.error);
        a.shape.chunk = logit_chunk(P, steps);
        a.shape.b_mn = first;
        a.tok = tok;
        a.lse = lse;
        a.rest = rest;
        a.wmax = wmax;
        a.g = g;
        a.low = terms > 1 ? g + static_cast<size_t>(c.T) * piece : nullptr;
        a.ldg = piece;
        a.first = first;
        a.count = count;
        if (kept) {
            const dim3 grid(static_cast<unsigned>(ceil_div(count, kFewColumns)), static_cast<unsigned>(c.T));
            e = gemm::launch_early(few_kernel<T>, grid, kFewThreads, 0, 1, stream, tok, logits.first.args.z, logits.first.args.ldz, part,
                                   2 * ceil_div(c.N, kTN), logits.first.args.target, c.loss, c.lse, c.rest, rows, g, a.low, piece);
        } else {
            e = gemm::launch(pieces, stream);
        }
        if (e != cudaSuccess) return e;
        gemm::Jobs<Hidden<T>, Head<T>> both = {};
        if (dh) {
            using L = typename Hidden<T>::Layout;
            auto& job = both.first;
            if ((e = gemm::encode_operand<L, false>(&job.map_a, g, all_rows, count, static_cast<uint64_t>(piece) * 2, gemm::kRows)) != cudaSuccess) return e;
            if ((e = gemm::encode_operand<L, true>(&job.map_b, c.head, c.K, c.N, c.ld_head * 2, 0)) != cudaSuccess) return e;
            auto& b = job.args;
            b.shape = tiles_h;
            b.shape.steps = ceil_div(count, L::kK);
            b.shape.splits = ceil_div(b.shape.steps, tiles_h.split_steps);
            b.shape.b_k = first;
            b.T_ = all_rows;
            b.K = c.K;
            b.sum = sum;
            b.parts = reinterpret_cast<float*>(ws + sp.parts);
            b.add = first > 0;
            if (direct) b.out = static_cast<T*>(c.dhidden);
            b.ld = c.ld_dhidden;
            b.wmax = wmax;
            b.tok = tok;
            if (first == 0) splits = b.shape.splits;
        }
        if (dw) {
            using L = typename Head<T>::Layout;
            auto& job = both.second;
            if ((e = gemm::encode_operand<L, true>(&job.map_a, g, count, all_rows, static_cast<uint64_t>(piece) * 2, 0)) != cudaSuccess) return e;
            if ((e = gemm::encode_operand<L, true>(&job.map_b, hidden, c.K, all_rows, static_cast<uint64_t>(c.K) * 2, 0)) != cudaSuccess) return e;
            auto& b = job.args;
            b.shape = head_parts != nullptr ? tiles_w : gemm::whole_tiles(ceil_div(count, kTM), ceil_div(c.K, kTN), ceil_div(all_rows, L::kK), c.error);
            b.parts = head_parts;
            b.rows = count;
            b.K = c.K;
            b.wmax = wmax;
            b.out = static_cast<T*>(c.dhead) + static_cast<size_t>(first) * c.ld_dhead;
            b.ld = c.ld_dhead;
            b.wide = reinterpret_cast<uintptr_t>(c.dhead) % 32 == 0 && c.K % 16 == 0 && c.ld_dhead % 16 == 0;
        }
        both.first.args.shape.error = c.error;   // (one gradient alone: the other has no tiles)
        if ((e = gemm::launch(both, stream)) != cudaSuccess) return e;
    }
    const bool sum_dh = dh && !direct;
    if (sum_dh || head_parts != nullptr) {
        Sums sums = {};
        if (sum_dh) {
            sums.elements = static_cast<size_t>(c.T) * (c.K / 8);
            sums.sum = sum;
            sums.parts = reinterpret_cast<float*>(ws + sp.parts);
            sums.tiles_m = tiles_h.tiles_m;
            sums.tiles_n = tiles_h.tiles_n;
            sums.whole = tiles_h.whole;
            sums.splits = splits;
            sums.terms = terms;
            sums.out = c.dhidden;
            sums.ld = c.ld_dhidden;
        }
        if (head_parts != nullptr) {
            sums.head = tiles_w;
            sums.head_parts = head_parts;
            sums.head_out = c.dhead;
            sums.head_ld = c.ld_dhead;
            sums.head_rows = c.N;
        }
        const size_t total = sums.elements + static_cast<size_t>(sums.head.tiles()) * (kTM * kTN / 8);
        const size_t want = (total + 255) / 256, cap = static_cast<size_t>(sm_count()) * 8;
        // (not early: a product's CTA leaves no registers for this kernel's, which would all start on the few SMs
        // that are through first: 100 x 64,026 x 2,560 241 us, 231)
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(want < cap ? want : cap));
        cfg.blockDim = dim3(256);
        cfg.stream = stream;
        if ((e = cudaLaunchKernelEx(&cfg, sum_kernel<T>, tok, sums, c.K, wmax)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <class T>
cudaError_t run_typed(const CrossEntropyArgs& c, cudaStream_t stream) {
    return c.T <= gemm::kRows ? run<T, 1>(c, stream) : run<T, 2>(c, stream);
}

}  // namespace ce

size_t cross_entropy_workspace_bytes(int T, int N, int K, bool loss, bool dhidden, bool dhead, bool two_terms) {
    return ce::space_of(T, N, K, loss, dhidden, dhead, two_terms).bytes;
}

cudaError_t launch_cross_entropy(const CrossEntropyArgs& a, cudaStream_t s) {
    return a.type == DH_T_F16 ? ce::run_typed<__half>(a, s) : ce::run_typed<__nv_bfloat16>(a, s);
}

}  // namespace dh
