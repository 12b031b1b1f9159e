// FP8 (E4M3) product with one scale per block of 128: y = x W'^T, and the gradient in its
// input, dx = dy W'.
//
//   activations, per token and 128 features: s = max(amax, 1e-12) / 448,
//     c = E4M3_RNE(clamp(x / s, +-448));  weights the same per 128 x 128 block;
//   y_mn = sum_b sx_mb sw_(n/128)b sum_(k in b) cx_mk cw_nk,
//   dx_mk = sum_b sdy_mb sw_b(k/128) sum_(n in b) cdy_mn cw_nk.
// The inner sums run on the tensor cores (kind::f8f6f4, exact products, 32-bit accumulators);
// 128 is one stage of K (dh_gemm.cuh), so each step leaves an accumulator of its own, which the
// epilogue multiplies by the two scales and adds to 32-bit sums in registers.
//
// The product of many tokens is bound by that hand-over (dh_gemm.cuh): 8,192 x 64,026 x 2,560 takes
// 1,150 us (2,330 TFLOP/s; 710 us at twice the measured bf16 rate), its quantiser about 20 of them; the
// gradient of 4,096 x 4,608 x 2,560 54.4. Few tokens: dh_fp8_few.cuh.
#include "dh_fp8_blocks.cuh"

namespace dh {
namespace f8 {

using gemm::Acc;
using gemm::ceil_div;
using gemm::Tile;

// ------------------------------------------------------------ quantisation ----

// Codes and scales of rows x [M][width]: eight lanes per block of 128, 16 elements each.
// codes [M][ldc] (ldc = width rounded up to 16, zeros beyond width), scales [blocks][M].
constexpr int kQThreads = 256;
template <class T, bool VEC>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const T* x, long long ldx, int M, int width, uint8_t* codes, int ldc,
                                                             float* scales) {
    programmatic_wait();
    const unsigned per_row = static_cast<unsigned>(ceil_div(width, kBlock));
    const unsigned unit = blockIdx.x * (kQThreads / 8) + (threadIdx.x >> 3);   // < 2^31 (checked)
    const unsigned m = unit / per_row, b = unit - m * per_row;
    const bool in = m < static_cast<unsigned>(M);
    const int k = static_cast<int>(b) * kBlock + (threadIdx.x & 7) * 16, n = in ? min(16, width - k) : 0;
    uint4 w;
    const float s = encode16<T, VEC>(Rows<T>{x, ldx, M, width}, static_cast<int>(m), k, n, w);
    if (in && (threadIdx.x & 7) == 0) scales[static_cast<size_t>(b) * M + m] = s;
    if (n > 0) *reinterpret_cast<uint4*>(codes + static_cast<size_t>(m) * ldc + k) = w;
}

// A weight's blocks: one CTA per 128 x 128, its 16,384 values in registers between the maximum
// and the codes. Rows W[idx[n]]; an id outside [0, V) leaves its row and sets the error word.
constexpr int kWThreads = 256;
__global__ void __launch_bounds__(kWThreads) blocks_kernel(const uint16_t* __restrict__ W, int V, int K, const int32_t* __restrict__ idx,
                                                           int N, uint8_t* __restrict__ q, float* __restrict__ scale, Workspace* ws) {
    const int nb = blockIdx.x, kb = blockIdx.y, piece = threadIdx.x & 15, k = kb * kBlock + piece * 8;   // 8 values of a row
    uint4 v[8];
    uint32_t there = 0;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = nb * kBlock + i * 16 + (threadIdx.x >> 4);
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (n >= N || k >= K) continue;
        const int id = idx[n];
        if (id < 0 || id >= V) {
            atomicOr(&ws->error, kDevErrIdx);
            continue;
        }
        there |= 1u << i;
        v[i] = *reinterpret_cast<const uint4*>(W + static_cast<size_t>(id) * K + k);
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    __shared__ float s_top[kWThreads / 32];
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
    top = s_top[0];
#pragma unroll
    for (int i = 1; i < kWThreads / 32; ++i) top = fmaxf(top, s_top[i]);
    const float s = act_fp8_scale(top);
    if (threadIdx.x == 0) scale[static_cast<size_t>(nb) * gridDim.y + kb] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!(there >> i & 1u)) continue;
        const int n = nb * kBlock + i * 16 + (threadIdx.x >> 4);
        *reinterpret_cast<uint2*>(q + static_cast<size_t>(n) * K + k) =
            make_uint2(act_fp8_pair(v[i].x, s) | (act_fp8_pair(v[i].y, s) << 16), act_fp8_pair(v[i].z, s) | (act_fp8_pair(v[i].w, s) << 16));
    }
}

// ----------------------------------------------------------------- product ----

// 32 results of a row at `out`, 32-byte aligned, `valid` of them wanted.
template <class TY>
__device__ __forceinline__ void store_row(TY* out, const float* v, int valid) {
    constexpr int kPer = 32 / sizeof(TY);   // results in 32 bytes
#pragma unroll
    for (int i = 0; i < 32; i += kPer) {
        if (valid >= i + kPer) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (sizeof(TY) == 2) w[j] = rows::Elem<TY>::pack2(v[i + 2 * j], v[i + 2 * j + 1]);
                else w[j] = __float_as_uint(v[i + j]);
            }
            store32(out + i, w);
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (i + j < valid) out[i + j] = rows::Elem<TY>::store(v[i + j]);
        }
    }
}

// A warp's 32 x 32 words, lane r's v[c] to lane c's v[r]: five exchanges between lanes (and
// words) that differ in one bit.
__device__ __forceinline__ void transpose32(uint32_t* v, int lane) {
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) {
        const bool up = (lane & b) != 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i & b) continue;
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, up ? v[i] : v[i | b], b);
            if (up) v[i] = other;
            else v[i | b] = other;
        }
    }
}

// How rows of results lie: whole 32-byte pieces, whole 32-bit words, or at any address.
enum RowAlign { kAny, kWords, kPieces };

// A warp's results, 64 columns of 32 rows (lane = row; `rows` of them wanted, `valid` columns),
// to the row-major y of its first row. Rows in whole 32-byte pieces: each lane its own. Others:
// transposed, so that the lanes store neighbouring words (or, at odd addresses of 16-bit types,
// elements).
template <class TY>
__device__ __forceinline__ void store64(TY* y, long long ldy, const float (&v)[64], int rows_, int valid, int align, int lane) {
    if (align == kPieces) {
        if (lane < rows_) {
#pragma unroll
            for (int c = 0; c < 64; c += 32) store_row<TY>(y + lane * ldy + c, v + c, valid - c);
        }
    } else if (sizeof(TY) == 2 && align == kWords) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if constexpr (sizeof(TY) == 2) w[i] = rows::Elem<TY>::pack2(v[2 * i], v[2 * i + 1]);
        transpose32(w, lane);
        y += 2 * lane;
        const int left = valid - 2 * lane;
#pragma unroll
        for (int i = 0; i < 32; ++i, y += ldy) {
            if (i < rows_ && left > 1) *reinterpret_cast<uint32_t*>(y) = w[i];
            else if (i < rows_ && left > 0) *reinterpret_cast<uint16_t*>(y) = static_cast<uint16_t>(w[i]);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[c + i]);
            transpose32(w, lane);
            TY* out = y + c + lane;
            const int left = valid - c - lane > 0 ? rows_ : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i, out += ldy)
                if (i < left) *out = rows::Elem<TY>::store(__uint_as_float(w[i]));
        }
    }
}

// Tokens along the rows of a tile, output features along its columns; W K-major for y, and
// MN-major (its rows along the contraction) for dx.
template <class TY, bool GRADIENT, int TN>
struct Product {
    using Layout = gemm::Layout<1, TN, 1, false, GRADIENT, TN / 16, 2>;
    static constexpr int kFormat = 0;
    static constexpr int kChunk = 1;
    static constexpr bool kAKeep = true, kBKeep = true;
    struct Args {
        gemm::Shape shape;
        const float* sx;      // [steps][M]
        const float* sw;      // scale of output block j and step b at j * sw_j + b * sw_b
        int sw_j, sw_b;
        int M, N;             // tokens, output features
        TY* y;
        long long ldy;
        int align;            // RowAlign of y
        float* parts;         // sums of the tiles in parts, [split][M][ldp], or, behind whole tiles (ldp 0),
        int ldp;              // [split][tile][128][TN]
    };
    __device__ static bool tile(const Args& a, const Tile& t, int warp, int lane, int, Acc<Layout>& acc) {
        constexpr int kPart = Layout::kPart;
        static_assert(kPart == 64 && Layout::kP == 1, "a warp's columns lie in one block of the weight");
        const int row0 = t.m * gemm::kRows + (warp & 3) * 32, row = row0 + lane, steps = t.steps;
        const int n0 = t.n * Layout::kTN + (warp >> 2) * kPart;
        const bool in = row < a.M;
        // (columns beyond N: any scale)
        const float* sw = a.sw + static_cast<size_t>(n0 < a.N ? n0 / kBlock : 0) * a.sw_j + static_cast<size_t>(t.k0) * a.sw_b;
        const float* sx = a.sx + static_cast<size_t>(t.k0) * a.M + (in ? row : 0);
        float sum[kPart];
#pragma unroll
        for (int i = 0; i < kPart; ++i) sum[i] = 0.0f;
        const auto scale_at = [&](int b) {
            b = b < steps ? b : steps - 1;
            return make_float2(sx[static_cast<size_t>(b) * a.M], __ldg(sw + static_cast<size_t>(b) * a.sw_b));
        };
        float2 s1 = scale_at(0), s2 = scale_at(1);   // two steps ahead: a load takes longer than a step
#pragma unroll 1
        for (int b = 0; b < steps; ++b) {
            const float s = s1.x * s1.y;
            s1 = s2;
            s2 = scale_at(b + 2);
            const uint32_t at = acc.next();
            if (at == ~0u) return false;
            const uint32_t from = at + (static_cast<uint32_t>(warp & 3) << 21) + (warp >> 2) * kPart;
#pragma unroll
            for (int c = 0; c < kPart; c += 16) {
                uint32_t r[16];
                tc::tmem_load16(from + c, r);
                tc::tmem_load_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[c + i] = fmaf(s, __uint_as_float(r[i]), sum[c + i]);
            }
            acc.release();
        }
        if (t.split >= 0) {
            size_t to = (static_cast<size_t>(t.split) * a.M + row0) * a.ldp + n0;
            if (a.ldp == 0) {
                const int rest = a.shape.tiles() - a.shape.whole, at = gemm::tile_index(a.shape.tiles_m, a.shape.tiles_n, t.m, t.n) - a.shape.whole;
                to = ((static_cast<size_t>(t.split) * rest + at) * gemm::kRows + (warp & 3) * 32) * TN + (warp >> 2) * kPart;
            }
            if (n0 < a.N) store64<float>(a.parts + to, a.ldp == 0 ? TN : a.ldp, sum, a.M - row0, a.N - n0, kPieces, lane);
        } else if (n0 < a.N) store64<TY>(a.y + static_cast<size_t>(row0) * a.ldy + n0, a.ldy, sum, a.M - row0, a.N - n0, a.align, lane);
        __syncwarp();
        return true;
    }
};

// y from the sums of its parts, in order, where all tiles are in parts.
template <class TY>
__global__ void __launch_bounds__(256) sum_kernel(const float* parts, int splits, int M, int N, int ldp, TY* y, long long ldy) {
    programmatic_wait();
    const unsigned n = blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n >= static_cast<unsigned>(N)) return;
    const float* p = parts + static_cast<size_t>(m) * ldp + n;
    float v = *p;
#pragma unroll 4
    for (int s = 1; s < splits; ++s) v += p[static_cast<size_t>(s) * M * ldp];
    y[static_cast<size_t>(m) * ldy + n] = rows::Elem<TY>::store(v);
}

// The same for the tiles behind whole ones: 512 elements of a tile per CTA. (In the layout of whole
// planes those would take [split][M][N]; where all tiles are in parts, that one is the shorter:
// 300 x 1,024 x 2,560 8.2 us, 10.0 tile by tile.)
constexpr int kSumElements = 512;
template <class TY, int TN>
__global__ void __launch_bounds__(256) rest_kernel(const float* parts, gemm::Shape shape, int M, int N, TY* y, long long ldy) {
    programmatic_wait();
    constexpr unsigned per = gemm::kRows * TN / kSumElements;
    const unsigned at = blockIdx.x / per, first = (blockIdx.x - at * per) * kSumElements + threadIdx.x;
    const int index = shape.whole + static_cast<int>(at);
    const size_t step = static_cast<size_t>(shape.tiles() - shape.whole) * (gemm::kRows * TN);
    shape.whole = shape.tiles();
    const Tile t = gemm::tile_at(shape, index);
    const float* p = parts + static_cast<size_t>(at) * (gemm::kRows * TN) + first;
    constexpr int kEach = kSumElements / 256;
    float v[kEach] = {};
    bool in[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) in[i] = t.m * gemm::kRows + static_cast<int>((first + i * 256) / TN) < M;
#pragma unroll 4
    for (int s = 0; s < shape.splits; ++s) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) v[i] += in[i] ? p[s * step + i * 256] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int m = t.m * gemm::kRows + static_cast<int>((first + i * 256) / TN), n = t.n * TN + static_cast<int>((first + i * 256) % TN);
        if (in[i] && n < N) y[static_cast<size_t>(m) * ldy + n] = rows::Elem<TY>::store(v[i]);
    }
}

// ------------------------------------------------------------------- host ----

int part_stride(int out) { return (out + 7) / 8 * 8; }

// How a product of many tokens runs: the width of its tiles, the tiles that are multiplied whole,
// and the parts of the contraction of the others, which fill a round over the SMs.
struct Plan {
    int tn, whole, parts, part_steps;
    float us;
    int tiles(int M, int out) const { return ceil_div(M, gemm::kRows) * ceil_div(out, tn); }
    size_t part_bytes(int M, int out) const {
        if (parts == 1) return 0;
        if (whole == 0) return static_cast<size_t>(parts) * M * part_stride(out) * sizeof(float);
        return static_cast<size_t>(parts) * (tiles(M, out) - whole) * (gemm::kRows * tn) * sizeof(float);
    }
};

// By rounds of tiles over the SMs times a step's time, or by reading the weight. A step takes
// 0.43 us in a 256-wide tile, 0.38 in a 128-wide one: wide tiles have twice the work between two
// hand-overs, narrow ones spread a small product over more SMs (512 x 4,608 x 2,560 15.0 wide,
// 13.3 narrow). With one row block, which alone reads its columns of the weight, 0.67 and 0.40 (1 x
// 20,000 x 2,560 17). Parts cost a second kernel: 200 tokens, gradient of 64,026 x 2,560 193 in one
// part, 55 in sixteen.
Plan plan_of(int M, int out, int width) {
    const int steps = ceil_div(width, kBlock);
    Plan best = {};
    constexpr struct { int tn; float step, alone; } kForms[] = {{256, 0.43f, 0.67f}, {128, 0.38f, 0.40f}};
    for (const auto& f : kForms) {
        const long long tiles = static_cast<long long>(ceil_div(M, gemm::kRows)) * ceil_div(out, f.tn), rest = tiles % kSms;
        const float step = M <= gemm::kRows ? f.alone : f.step, tile = steps * step + 1.0f, full = static_cast<float>(tiles / kSms) * tile;
        const float whole = full + (rest > 0 ? tile : 0.0f);
        if (best.tn == 0 || whole < best.us) best = {f.tn, static_cast<int>(tiles), 1, steps, whole};
        const float most = static_cast<float>(M) * out, there = static_cast<float>(rest) * (gemm::kRows * f.tn);
        for (int p = 2; rest > 0 && p <= 16 && steps / p >= 4; ++p) {
            const int part = ceil_div(steps, p);
            const float us = full + static_cast<float>((rest * p + kSms - 1) / kSms) * (part * step + 1.0f) + 2.0f +
                             p * (there < most ? there : most) * 1.0e-6f;
            if (us < best.us) best = {f.tn, static_cast<int>(tiles - rest), ceil_div(steps, part), part, us};
        }
    }
    const float read = static_cast<float>(width) * out * (1.0f / 4.4e6f);
    if (best.us < read) best.us = read;
    best.us += 2.5f;   // quantising before it
    return best;
}

template <class T>
cudaError_t quantize(const Fp8BlockArgs& f, int width, uint8_t* codes, int ldc, float* scales, cudaStream_t s) {
    const bool vec = rows_aligned16(f.x, f.ldx * static_cast<long long>(sizeof(T)), f.M);
    const unsigned units = static_cast<unsigned>(f.M) * static_cast<unsigned>(ceil_div(width, kBlock));
    const unsigned grid = (units + kQThreads / 8 - 1) / (kQThreads / 8);
    return gemm::launch_early(vec ? quantize_kernel<T, true> : quantize_kernel<T, false>, dim3(grid), kQThreads, 0, 1, s,
                              static_cast<const T*>(f.x), f.ldx, f.M, width, codes, ldc, scales);
}

template <class TY, bool GRADIENT, int TN>
cudaError_t product(const Fp8BlockArgs& f, const Plan& plan, const uint8_t* codes, int ldc, const float* scales, float* parts, cudaStream_t s) {
    using P = Product<TY, GRADIENT, TN>;
    using L = typename P::Layout;
    const int width = GRADIENT ? f.N : f.K, out = GRADIENT ? f.K : f.N, kb = ceil_div(f.K, kBlock);
    gemm::Jobs<P> jobs = {};
    cudaError_t e = gemm::encode_operand<L, false>(&jobs.first.map_a, codes, f.M, width, ldc, gemm::kRows);
    if (e != cudaSuccess) return e;
    if ((e = gemm::encode_operand<L, GRADIENT>(&jobs.first.map_b, f.q, out, width, f.K, L::kBRows)) != cudaSuccess) return e;
    typename P::Args& a = jobs.first.args;
    const int steps = ceil_div(width, kBlock);
    a.shape = gemm::whole_tiles(ceil_div(f.M, gemm::kRows), ceil_div(out, L::kTN), steps, f.error);
    a.shape.rounds = f.probe_rounds;
    a.shape.idle = f.probe_role;
    a.sx = scales;
    a.sw = f.scale;
    a.sw_j = GRADIENT ? 1 : kb;
    a.sw_b = GRADIENT ? kb : 1;
    a.M = f.M;
    a.N = out;
    a.y = static_cast<TY*>(f.y);
    a.ldy = f.ldy;
    const uintptr_t at = reinterpret_cast<uintptr_t>(f.y) | (f.M == 1 ? 0 : static_cast<uintptr_t>(f.ldy) * sizeof(TY));
    a.align = at % 32 == 0 ? kPieces : at % 4 == 0 ? kWords : kAny;
    if (plan.parts == 1) return gemm::launch(jobs, s);
    a.shape.whole = plan.whole;
    a.shape.splits = plan.parts;
    a.shape.split_steps = plan.part_steps;
    a.parts = parts;
    a.ldp = plan.whole == 0 ? part_stride(out) : 0;
    if ((e = gemm::launch(jobs, s)) != cudaSuccess) return e;
    if (plan.whole == 0) {
        const dim3 grid(static_cast<unsigned>(ceil_div(out, 256)), static_cast<unsigned>(f.M));   // (M: rows of less than kSms tiles)
        return gemm::launch_early(sum_kernel<TY>, grid, 256, 0, 1, s, parts, plan.parts, f.M, out, a.ldp, a.y, a.ldy);
    }
    const dim3 grid(static_cast<unsigned>(a.shape.tiles() - plan.whole) * (gemm::kRows * TN / kSumElements));   // (less than kSms tiles)
    return gemm::launch_early(rest_kernel<TY, TN>, grid, 256, 0, 1, s, parts, a.shape, f.M, out, a.y, a.ldy);
}

template <class TY>
cudaError_t run_many(const Fp8BlockArgs& f, const Plan& p, const uint8_t* codes, int ldc, const float* scales, float* parts, cudaStream_t s) {
    const auto with = [&](auto tn) {
        constexpr int kTN = decltype(tn)::value;
        return f.gradient ? product<TY, true, kTN>(f, p, codes, ldc, scales, parts, s)
                          : product<TY, false, kTN>(f, p, codes, ldc, scales, parts, s);
    };
    return p.tn == 128 ? with(std::integral_constant<int, 128>()) : with(std::integral_constant<int, 256>());
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Whether a product takes the form of few tokens: where it is estimated shorter, and up to 16 also where
// it is up to 4 us longer (one or two launches for two or three: 16 x 2,560 x 5,120 9.0 us and 8.6, but 11
// and 15 as calls). Measured, us (few / many): 32 x 64,026 x 2,560 33 / 42, 64 37 / 37; 32 x 4,608 x 2,560
// 9.1 / 8.5, 64 10.1 / 8.7.
bool take_few(int M, int out, int width, FewPlan* few, Plan* many) {
    *few = few_plan(M, out, width);
    *many = plan_of(M, out, width);
    return few->splits > 0 && few->us <= many->us + (M <= 16 ? 4.0f : 0.0f);
}

template <class TY>
cudaError_t run(const Fp8BlockArgs& f, cudaStream_t s) {
    const int width = f.gradient ? f.N : f.K, out = f.gradient ? f.K : f.N, ldc = ceil_div(width, 16) * 16;
    FewPlan few;
    Plan p;
    const bool use_few = take_few(f.M, out, width, &few, &p);
    if (use_few && few.fused) return launch_few<TY>(f, few, nullptr, 0, nullptr, s);
    uint8_t* codes = static_cast<uint8_t*>(f.ws);
    float* scales = reinterpret_cast<float*>(codes + up256(static_cast<size_t>(f.M) * ldc));
    float* parts = reinterpret_cast<float*>(codes + up256(static_cast<size_t>(f.M) * ldc) +
                                            up256(static_cast<size_t>(f.M) * ceil_div(width, kBlock) * sizeof(float)));
    const cudaError_t e = f.x_type == DH_T_BF16  ? quantize<__nv_bfloat16>(f, width, codes, ldc, scales, s)
                          : f.x_type == DH_T_F16 ? quantize<__half>(f, width, codes, ldc, scales, s)
                                                 : quantize<float>(f, width, codes, ldc, scales, s);
    if (e != cudaSuccess) return e;
    if (use_few) return launch_few<TY>(f, few, codes, ldc, scales, s);
    return run_many<TY>(f, p, codes, ldc, scales, parts, s);
}

}  // namespace f8

size_t fp8_block_workspace_bytes(int M, int width, int out) {
    f8::FewPlan few;
    f8::Plan many;
    const bool use_few = f8::take_few(M, out, width, &few, &many);
    if (use_few && few.fused) return DH_WORKSPACE_ALIGN;   // not used
    return f8::up256(static_cast<size_t>(M) * (f8::ceil_div(width, 16) * 16)) +
           f8::up256(static_cast<size_t>(M) * f8::ceil_div(width, f8::kBlock) * sizeof(float)) +
           (use_few ? 0 : f8::up256(many.part_bytes(M, out)));
}

cudaError_t launch_fp8_quantize_blocks(const uint16_t* W, int V, int K, const int32_t* idx, int N, uint8_t* q, float* scale, Workspace* ws,
                                       cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(f8::ceil_div(N, f8::kBlock)), static_cast<unsigned>(f8::ceil_div(K, f8::kBlock)));
    f8::blocks_kernel<<<grid, f8::kWThreads, 0, s>>>(W, V, K, idx, N, q, scale, ws);
    return cudaGetLastError();
}

cudaError_t launch_fp8_blocks(const Fp8BlockArgs& f, cudaStream_t s) {
    switch (f.y_type) {
        case DH_T_BF16: return f8::run<__nv_bfloat16>(f, s);
        case DH_T_F16: return f8::run<__half>(f, s);
        default: return f8::run<float>(f, s);
    }
}

}  // namespace dh
