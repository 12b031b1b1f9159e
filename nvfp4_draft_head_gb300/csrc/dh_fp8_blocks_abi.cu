// C-ABI entry points of the FP8 block-scaled product: argument checks on the host, then the
// launches of dh_fp8_blocks.cu. See include/drafthead.h.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/drafthead.h"
#include "dh_common.cuh"
#include "dh_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? DH_OK : dh::record_cuda_error(e); }

int type_bytes(int type) { return type == DH_T_BF16 || type == DH_T_F16 ? 2 : type == DH_T_F32 ? 4 : 0; }

constexpr int kMaxN = 1 << 24, kMaxK = 1 << 20, kMaxM = 1 << 24;

bool weight_ok(int N, int K) { return N >= 1 && N <= kMaxN && K >= 16 && K <= kMaxK && K % 16 == 0; }

bool tokens_ok(int M, int width, int out) {
    return M >= 1 && M <= kMaxM && width >= 1 && width <= kMaxN && out >= 1 && out <= kMaxN &&
           static_cast<int64_t>(M) * ((width + 127) / 128) < (1ll << 31) &&
           ((static_cast<int64_t>(M) + 127) / 128) * ((out + 127) / 128) <= (1 << 30);
}

int product(const dh_fp8_blocks_t* w, bool gradient, const void* x, int x_type, int64_t ldx, int M, void* y, int y_type, int64_t ldy,
            void* ws, size_t ws_bytes, unsigned int* error, void* stream, int probe_role = 0, unsigned int probe_rounds = 0) {
    if (w == nullptr || w->q == nullptr || w->scale == nullptr || x == nullptr || y == nullptr) return DH_ERR_ARG;
    if (type_bytes(x_type) == 0 || type_bytes(y_type) == 0 || x == y) return DH_ERR_ARG;   // (not in place)
    if (!weight_ok(w->N, w->K)) return DH_ERR_SHAPE;
    const int width = gradient ? w->N : w->K, out = gradient ? w->K : w->N;
    if (!tokens_ok(M, width, out)) return DH_ERR_SHAPE;
    if (M > 1 && (ldx < width || ldy < out)) return DH_ERR_SHAPE;
    if (!aligned(w->q, 16) || !aligned(w->scale, 4) || !aligned(x, type_bytes(x_type)) || !aligned(y, type_bytes(y_type)) || !aligned(error, 4))
        return DH_ERR_ALIGN;
    if (ws == nullptr) return DH_ERR_ARG;
    if (!aligned(ws, DH_WORKSPACE_ALIGN) || ws_bytes < dh::fp8_block_workspace_bytes(M, width, out)) return DH_ERR_WORKSPACE;
    dh::Fp8BlockArgs a = {};
    a.q = static_cast<const uint8_t*>(w->q);
    a.scale = w->scale;
    a.N = w->N;
    a.K = w->K;
    a.M = M;
    a.gradient = gradient;
    a.x = x;
    a.x_type = x_type;
    a.ldx = ldx;
    a.y = y;
    a.y_type = y_type;
    a.ldy = ldy;
    a.ws = ws;
    a.error = error;
    a.probe_role = probe_role;
    a.probe_rounds = probe_rounds;
    return cuda_status(dh::launch_fp8_blocks(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int fp8_quantize_blocks(const void* W, int V, int K, const int32_t* idx, int N, uint8_t* q, float* scale, void* ws, size_t ws_bytes,
                        void* stream) {
    if (W == nullptr || idx == nullptr || q == nullptr || scale == nullptr || ws == nullptr) return DH_ERR_ARG;
    if (V < 1 || !weight_ok(N, K)) return DH_ERR_SHAPE;
    if (!aligned(W, 16) || !aligned(idx, 4) || !aligned(q, 16) || !aligned(scale, 4)) return DH_ERR_ALIGN;
    if (!aligned(ws, DH_WORKSPACE_ALIGN) || ws_bytes < dh::kWorkspaceHeader) return DH_ERR_WORKSPACE;
    return cuda_status(dh::launch_fp8_quantize_blocks(static_cast<const uint16_t*>(W), V, K, idx, N, q, scale, static_cast<dh::Workspace*>(ws),
                                                      static_cast<cudaStream_t>(stream)));
}

size_t fp8_block_matmul_workspace_bytes(int M, int width, int out) {
    return tokens_ok(M, width, out) ? dh::fp8_block_workspace_bytes(M, width, out) : 0;
}

int fp8_block_matmul(const dh_fp8_blocks_t* w, const void* x, int x_type, int64_t ldx, int M, void* y, int y_type, int64_t ldy, void* ws,
                     size_t ws_bytes, unsigned int* error, void* stream) {
    return product(w, false, x, x_type, ldx, M, y, y_type, ldy, ws, ws_bytes, error, stream);
}

int fp8_block_matmul_input_gradient(const dh_fp8_blocks_t* w, const void* dy, int dy_type, int64_t lddy, int M, void* dx, int dx_type,
                                    int64_t lddx, void* ws, size_t ws_bytes, unsigned int* error, void* stream) {
    return product(w, true, dy, dy_type, lddy, M, dx, dx_type, lddx, ws, ws_bytes, error, stream);
}

int fp8_block_matmul_wait_probe(const dh_fp8_blocks_t* w, const void* x, int M, void* y, void* ws, size_t ws_bytes, int role,
                                unsigned int rounds, unsigned int* error, void* stream) {
    if (w == nullptr || error == nullptr || role < 0 || role > 2 || rounds < 1 || rounds > 4096) return DH_ERR_ARG;
    return product(w, false, x, DH_T_BF16, w->K, M, y, DH_T_BF16, w->N, ws, ws_bytes, error, stream, role, rounds);
}

}  // extern "C"
