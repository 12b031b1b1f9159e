// Softmax cross entropy of hidden states against a vocabulary given by its head rows, and
// its gradients, without logits in memory.
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
// the price of not keeping T x N probabilities.
//
// Roundings besides 32-bit arithmetic: g to the inputs' 16-bit type (the tensor cores take
// nothing wider from it; its error is that of rounding the results again), scaled by a power of
// two so that the largest row weight lies just under 1 (bf16) or 2^15 (f16, whose probabilities
// would be subnormal below 6e-5); the gradients once, at the end.
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

// 32 bytes, 32-byte aligned, in one store.
__device__ __forceinline__ void store32(void* p, const uint32_t* w) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
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
};

// The power of two by which row weights are scaled before g is rounded: the largest finite
// one's exponent (bits of |w|) is brought to -1, or to 14 for f16.
template <bool F16>
__device__ __forceinline__ int scale_exponent(uint32_t wmax) {
    const int e = static_cast<int>(wmax >> 23) - 127;   // floor(log2); -127 for subnormals and 0
    return (F16 ? 14 : -1) - (e < -100 ? -100 : e > 126 ? 126 : e);
}

// ---------------------------------------------------------------- the loss ----

template <class T>
struct Stats {
    using Layout = gemm::Layout<kPair, kTN, 2, false, false>;
    static constexpr int kFormat = std::is_same<T, __half>::value ? 0 : 1;
    static constexpr bool kPerStep = false, kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        Tokens tok;
        float2* part;   // [2 tiles_n][T]: maximum and sum of 128 columns
        float* target;  // [T]: the token's logit
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * kPair + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf;
        const int y = row < a.tok.T ? a.tok.row(row) : -1;
        const uint32_t at = acc.next();
        if (at == ~0u) return false;
        const uint32_t from = at + (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        float m = kNegInf, s = 0.0f;
#pragma unroll 1
        for (int c = 0; c < kHalf && n0 + c < a.tok.N; c += 32) {
            uint32_t r[32];
            tc::tmem_load32(from + c, r);
            tc::tmem_load_wait();
            const int valid = a.tok.N - (n0 + c);
            if (valid < 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = i < valid ? r[i] : __float_as_uint(kNegInf);
            }
            float top[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) top[i] = __uint_as_float(r[i]);
#pragma unroll
            for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], __uint_as_float(r[i]));
            const float next = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            const float ref = next == kNegInf ? 0.0f : next;   // nothing above -inf yet
            float sum[4] = {s * exp2_approx((m - ref) * kLog2e), 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[i & 3] += exp2_approx((__uint_as_float(r[i]) - ref) * kLog2e);
            s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            m = next;
            const int j = y - (n0 + c);
            if (__any_sync(0xFFFFFFFFu, j >= 0 && j < 32)) {
                float z = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) z = i == j ? __uint_as_float(r[i]) : z;
                if (j >= 0 && j < 32) a.target[row] = z;
                __syncwarp();
            }
        }
        acc.release();
        if (row < a.tok.T) a.part[static_cast<size_t>(2 * t.n + half) * a.tok.T + row] = make_float2(m, s);
        return true;
    }
};

// Joins the parts: 32 tokens per CTA, its warps over the parts, then over the warps.
constexpr int kJoinWarps = 32;
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2), ref = top == kNegInf ? 0.0f : top;
    s = s * exp2_approx((m - ref) * kLog2e) + s2 * exp2_approx((m2 - ref) * kLog2e);
    m = top;
}
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Tokens tok, const float2* __restrict__ part, int parts,
                                                               const float* __restrict__ target, float* __restrict__ loss,
                                                               float* __restrict__ lse, float* __restrict__ rest) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x * 32 + lane;
    float m = kNegInf, s = 0.0f;
    if (t < tok.T)
        for (int j = warp; j < parts; j += kJoinWarps) {
            const float2 p = part[static_cast<size_t>(j) * tok.T + t];
            join(m, s, p.x, p.y);
        }
    __shared__ float2 all[kJoinWarps][33];
    all[warp][lane] = make_float2(m, s);
    __syncthreads();
    if (warp != 0 || t >= tok.T) return;
#pragma unroll 4
    for (int j = 1; j < kJoinWarps; ++j) join(m, s, all[j][lane].x, all[j][lane].y);
    const float ln = logf(s), sum = m + ln;
    if (loss != nullptr) {
        const float w = tok.w(t);
        loss[t] = w != 0.0f && tok.row(t) >= 0 ? w * (ln + (m - target[t])) : 0.0f;
    }
    if (lse != nullptr) lse[t] = sum;
    if (rest != nullptr) {   // what the sum rounded away (two-sum)
        const float b = sum - m;
        rest[t] = (m - (sum - b)) + (ln - b);
    }
}

// --------------------------------------------------------------- gradients ----

// The largest finite row weight in use (bits of its magnitude), and, where dW is wanted, the
// hidden states with zeros in the rows that are left out: their g is 0, but 0 times what a
// padding row may hold (infinities, NaN) is not.
template <class T>
__global__ void __launch_bounds__(128) rows_kernel(const Tokens tok, const T* __restrict__ h, long long ld, int K, T* __restrict__ out,
                                                   uint32_t* __restrict__ wmax) {
    const int t = blockIdx.x;
    const float w = tok.w(t);
    const bool live = w != 0.0f && tok.row(t) >= 0;
    if (threadIdx.x == 0 && live) {
        const uint32_t bits = __float_as_uint(w) & 0x7FFFFFFFu;
        if (bits < 0x7F800000u) atomicMax(wmax, bits);   // (a maximum: the order does not matter)
    }
    if (out == nullptr) return;
    const uint4* src = reinterpret_cast<const uint4*>(h + static_cast<size_t>(t) * ld);
    uint4* dst = reinterpret_cast<uint4*>(out + static_cast<size_t>(t) * K);
    for (int i = threadIdx.x; i < K / 8; i += blockDim.x) dst[i] = live ? src[i] : make_uint4(0u, 0u, 0u, 0u);
}

template <class T>
struct Weights {   // g of a piece
    using Layout = gemm::Layout<kPair, kTN, 2, false, false>;
    static constexpr bool kF16 = std::is_same<T, __half>::value;
    static constexpr int kFormat = kF16 ? 0 : 1;
    static constexpr bool kPerStep = false, kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        Tokens tok;
        const float* lse;
        const float* rest;      // or null
        const uint32_t* wmax;
        T* g;                   // [T][ldg], ldg a multiple of 256
        int ldg;
        int first, count;       // the piece's rows of the head
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * kPair + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
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
        const uint32_t at = acc.next();
        if (at == ~0u) return false;
        const uint32_t from = at + (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        T* out = a.g + static_cast<size_t>(row) * a.ldg + c0;
#pragma unroll 1
        for (int c = 0; c < kHalf && c0 + c < a.count; c += 32) {
            uint32_t r[32];
            tc::tmem_load32(from + c, r);
            tc::tmem_load_wait();
            const int j = y - (a.first + c0 + c);
            const bool hit = __any_sync(0xFFFFFFFFu, j >= 0 && j < 32);
            float g[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) g[i] = exp2_approx(((__uint_as_float(r[i]) - lse) - rest) * kLog2e);
            if (hit) {
#pragma unroll
                for (int i = 0; i < 32; ++i) g[i] = i == j ? g[i] - 1.0f : g[i];
            }
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = live ? rows::Elem<T>::pack2(g[2 * i] * w, g[2 * i + 1] * w) : 0u;
            if (row < a.tok.T) {
                store32(out + c, v);
                store32(out + c + 16, v + 8);
            }
            __syncwarp();
        }
        acc.release();
        return true;
    }
};

// dh: g (along the piece) times the piece's head rows, as 32-bit sums per part of the piece.
template <class T>
struct Hidden {
    using Layout = gemm::Layout<kPair, kTN, 2, false, true>;
    static constexpr int kFormat = std::is_same<T, __half>::value ? 0 : 1;
    static constexpr bool kPerStep = false, kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        int T_, K;
        float* sum;   // [splits][T][K]
        int add;      // to what earlier pieces left
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * kPair + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf;
        const uint32_t at = acc.next();
        if (at == ~0u) return false;
        const uint32_t from = at + (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        float* out = a.sum + (static_cast<size_t>(t.split) * a.T_ + row) * a.K + n0;
#pragma unroll 1
        for (int c = 0; c < kHalf && n0 + c < a.K; c += 32) {
            uint32_t r[32];
            tc::tmem_load32(from + c, r);
            tc::tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                if (row >= a.T_ || n0 + c + i >= a.K) break;
                if (a.add) {
                    const float4 p = *reinterpret_cast<const float4*>(out + c + i), q = *reinterpret_cast<const float4*>(out + c + i + 4);
                    const float o[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[i + j] = __float_as_uint(o[j] + __uint_as_float(r[i + j]));
                }
                store32(out + c + i, r + i);
            }
            __syncwarp();
        }
        acc.release();
        return true;
    }
};

// dW: the piece's g (along the tokens) times the hidden states, final.
template <class T>
struct Head {
    using Layout = gemm::Layout<kPair, kTN, 2, true, true>;
    static constexpr bool kF16 = std::is_same<T, __half>::value;
    static constexpr int kFormat = kF16 ? 0 : 1;
    static constexpr bool kPerStep = false, kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        int rows, K;             // head rows of the piece
        const uint32_t* wmax;
        T* out;                  // the piece's first row
        long long ld;
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int rank, Acc<Layout>& acc) {
        const int row = (t.m * kPair + rank) * gemm::kRows + (warp & 3) * 32 + lane, half = warp >> 2;
        const int n0 = t.n * kTN + half * kHalf;
        const float scale = exp2i(-scale_exponent<kF16>(*a.wmax));
        const uint32_t at = acc.next();
        if (at == ~0u) return false;
        const uint32_t from = at + (static_cast<uint32_t>(warp & 3) << 21) + half * kHalf;
        T* out = a.out + static_cast<size_t>(row) * a.ld + n0;
#pragma unroll 1
        for (int c = 0; c < kHalf && n0 + c < a.K; c += 32) {
            uint32_t r[32];
            tc::tmem_load32(from + c, r);
            tc::tmem_load_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                if (row >= a.rows || n0 + c + i >= a.K) break;
                uint32_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = rows::Elem<T>::pack2(__uint_as_float(r[i + 2 * j]) * scale, __uint_as_float(r[i + 2 * j + 1]) * scale);
                __stcg(reinterpret_cast<uint4*>(out + c + i), make_uint4(v[0], v[1], v[2], v[3]));
            }
            __syncwarp();
        }
        acc.release();
        return true;
    }
};

// dh from the sums of its parts: eight elements per thread, parts in order. Rows that are left
// out are zeros whatever the head holds.
template <class T>
__global__ void __launch_bounds__(256) sum_kernel(const Tokens tok, const float* __restrict__ sum, int parts, int K,
                                                  const uint32_t* __restrict__ wmax, T* __restrict__ out, long long ld) {
    const float scale = exp2i(-scale_exponent<std::is_same<T, __half>::value>(*wmax));
    const size_t per_row = K / 8, total = static_cast<size_t>(tok.T) * per_row, step = static_cast<size_t>(tok.T) * K;
    for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total; i += static_cast<size_t>(gridDim.x) * blockDim.x) {
        const float* p = sum + i * 8;
        float v[8] = {};
        for (int s = 0; s < parts; ++s, p += step) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
        }
        const size_t row = i / per_row, col = i % per_row * 8;
        const bool live = tok.w(static_cast<int>(row)) != 0.0f && tok.row(static_cast<int>(row)) >= 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = live ? v[j] * scale : 0.0f;
        *reinterpret_cast<uint4*>(out + row * ld + col) = rows::Elem<T>::pack(v);
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

// Parts of a piece's contraction for dh: enough to fill the pairs of SMs once, at least eight
// steps long.
void hidden_parts(int T, int K, int piece, int* parts, int* steps) {
    const int tiles = ceil_div(T, kTM) * ceil_div(K, kTN), all = ceil_div(piece, 64);
    int p = tiles < 76 ? 76 / tiles : 1;
    if (p > all / 8) p = all / 8 > 0 ? all / 8 : 1;
    *steps = ceil_div(all, p);
    *parts = ceil_div(all, *steps);
}

struct Space {
    size_t wmax, part, target, lse, rest, g, hidden, sum, bytes;
};
Space space_of(int T, int N, int K, bool loss, bool dh, bool dw) {
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
    if (dh || dw) s.g = take(t * piece_rows(T, N) * 2);
    if (dw) s.hidden = take(t * K * 2);
    if (dh) {
        int parts, steps;
        hidden_parts(T, K, piece_rows(T, N), &parts, &steps);
        s.sum = take(t * K * 4 * parts);
    }
    s.bytes = at;
    return s;
}

template <class T>
cudaError_t run(const CrossEntropyArgs& c, cudaStream_t stream) {
    const bool loss = c.loss != nullptr, dh = c.dhidden != nullptr, dw = c.dhead != nullptr;
    const Space sp = space_of(c.T, c.N, c.K, loss, dh, dw);
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    Tokens tok = {c.tokens, c.row_of, c.weight, c.V, c.T, c.N};
    uint32_t* wmax = reinterpret_cast<uint32_t*>(ws + sp.wmax);
    const int tiles_m = ceil_div(c.T, kTM);
    cudaError_t e;
    CUtensorMap map_h, map_w;
    using K1 = typename Stats<T>::Layout;
    if ((e = gemm::encode_operand<K1, false>(&map_h, c.hidden, c.T, c.K, c.ld_hidden * 2, gemm::kRows)) != cudaSuccess) return e;
    if ((e = gemm::encode_operand<K1, false>(&map_w, c.head, c.N, c.K, c.ld_head * 2, K1::kBRows)) != cudaSuccess) return e;
    const int steps = ceil_div(c.K, K1::kK);
    const float* lse = c.lse_in;
    const float* rest = c.rest_in;
    if (loss) {
        typename Stats<T>::Args a = {};
        a.shape = {tiles_m, ceil_div(c.N, kTN), 1, steps, steps, 0, 0, 0, 0, c.error, 0, 0};
        a.tok = tok;
        a.part = reinterpret_cast<float2*>(ws + sp.part);
        a.target = reinterpret_cast<float*>(ws + sp.target);
        if ((e = gemm::launch<Stats<T>>(map_h, map_w, a, stream)) != cudaSuccess) return e;
        float* l = c.lse != nullptr ? c.lse : reinterpret_cast<float*>(ws + sp.lse);
        float* r = c.rest != nullptr ? c.rest : reinterpret_cast<float*>(ws + sp.rest);
        join_kernel<<<ceil_div(c.T, 32), 32 * kJoinWarps, 0, stream>>>(tok, a.part, 2 * a.shape.tiles_n, a.target, c.loss, l, r);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        lse = l;
        rest = r;
    }
    if (!dh && !dw) return cudaSuccess;

    T* hidden = dw ? reinterpret_cast<T*>(ws + sp.hidden) : nullptr;
    if ((e = cudaMemsetAsync(wmax, 0, 4, stream)) != cudaSuccess) return e;
    rows_kernel<T><<<c.T, 128, 0, stream>>>(tok, static_cast<const T*>(c.hidden), c.ld_hidden, c.K, hidden, wmax);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int piece = piece_rows(c.T, c.N);
    int parts, part_steps;
    hidden_parts(c.T, c.K, piece, &parts, &part_steps);
    T* g = reinterpret_cast<T*>(ws + sp.g);
    float* sum = reinterpret_cast<float*>(ws + sp.sum);
    int filled = 0;   // parts of dh that hold sums
    for (int first = 0; first < c.N; first += piece) {
        const int count = c.N - first < piece ? c.N - first : piece;
        typename Weights<T>::Args a = {};
        a.shape = {tiles_m, ceil_div(count, kTN), 1, steps, steps, 0, 0, first, 0, c.error, 0, 0};
        a.tok = tok;
        a.lse = lse;
        a.rest = rest;
        a.wmax = wmax;
        a.g = g;
        a.ldg = piece;
        a.first = first;
        a.count = count;
        if ((e = gemm::launch<Weights<T>>(map_h, map_w, a, stream)) != cudaSuccess) return e;
        CUtensorMap map_a, map_b;
        if (dh) {
            using L = typename Hidden<T>::Layout;
            if ((e = gemm::encode_operand<L, false>(&map_a, g, c.T, count, static_cast<uint64_t>(piece) * 2, gemm::kRows)) != cudaSuccess) return e;
            if ((e = gemm::encode_operand<L, true>(&map_b, c.head, c.K, c.N, c.ld_head * 2, 0)) != cudaSuccess) return e;
            typename Hidden<T>::Args b = {};
            const int all = ceil_div(count, L::kK);
            b.shape = {tiles_m, ceil_div(c.K, kTN), ceil_div(all, part_steps), all, part_steps, 0, 0, 0, first, c.error, 0, 0};
            b.shape.a_k = 0;
            b.T_ = c.T;
            b.K = c.K;
            b.sum = sum;
            b.add = first > 0;
            if (first == 0) filled = b.shape.splits;
            if ((e = gemm::launch<Hidden<T>>(map_a, map_b, b, stream)) != cudaSuccess) return e;
        }
        if (dw) {
            using L = typename Head<T>::Layout;
            if ((e = gemm::encode_operand<L, true>(&map_a, g, count, c.T, static_cast<uint64_t>(piece) * 2, 0)) != cudaSuccess) return e;
            if ((e = gemm::encode_operand<L, true>(&map_b, hidden, c.K, c.T, static_cast<uint64_t>(c.K) * 2, 0)) != cudaSuccess) return e;
            typename Head<T>::Args b = {};
            const int all = ceil_div(c.T, L::kK);
            b.shape = {ceil_div(count, kTM), ceil_div(c.K, kTN), 1, all, all, 0, 0, 0, 0, c.error, 0, 0};
            b.rows = count;
            b.K = c.K;
            b.wmax = wmax;
            b.out = static_cast<T*>(c.dhead) + static_cast<size_t>(first) * c.ld_dhead;
            b.ld = c.ld_dhead;
            if ((e = gemm::launch<Head<T>>(map_a, map_b, b, stream)) != cudaSuccess) return e;
        }
    }
    if (dh) {
        const size_t total = static_cast<size_t>(c.T) * (c.K / 8), want = (total + 255) / 256, cap = static_cast<size_t>(sm_count()) * 8;
        sum_kernel<T><<<static_cast<unsigned>(want < cap ? want : cap), 256, 0, stream>>>(tok, sum, filled, c.K, wmax, static_cast<T*>(c.dhidden),
                                                                                      c.ld_dhidden);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ce

size_t cross_entropy_workspace_bytes(int T, int N, int K, bool loss, bool dhidden, bool dhead) {
    return ce::space_of(T, N, K, loss, dhidden, dhead).bytes;
}

cudaError_t launch_cross_entropy(const CrossEntropyArgs& a, cudaStream_t s) {
    return a.type == DH_T_F16 ? ce::run<__half>(a, s) : ce::run<__nv_bfloat16>(a, s);
}

}  // namespace dh
