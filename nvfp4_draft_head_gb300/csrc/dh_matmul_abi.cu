// C-ABI entry points of the many-token NVFP4 product: argument checks on the
// host, then the launches of dh_matmul.cu. See include/drafthead.h.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/drafthead.h"
#include "dh_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? DH_OK : dh::record_cuda_error(e); }

int type_bytes(int type) { return type == DH_T_BF16 || type == DH_T_F16 ? 2 : type == DH_T_F32 ? 4 : 0; }

constexpr int kMaxN = 1 << 24, kMaxK = 1 << 20, kMaxM = 1 << 24;

int check_shape(int N, int K) {
    return N < 1 || K < 1 || N % 64 != 0 || K % 16 != 0 || N > kMaxN || K > kMaxK ? DH_ERR_SHAPE : DH_OK;
}

// The checks of a product's arguments; fills `a` where they pass.
int check_matmul(const dh_matmul_t* w, const void* x, int x_type, int64_t ldx, int M, void* y, int y_type, int64_t ldy,
                 void* ws, size_t ws_bytes, unsigned int* error, dh::MatmulArgs& a) {
    if (w == nullptr || w->packed == nullptr || w->scale == nullptr || x == nullptr || y == nullptr) return DH_ERR_ARG;
    if (type_bytes(x_type) == 0 || type_bytes(y_type) == 0) return DH_ERR_ARG;
    if (check_shape(w->N, w->K) != DH_OK || M < 1 || M > kMaxM) return DH_ERR_SHAPE;
    if (M > 1 && (ldx < w->K || ldy < w->N)) return DH_ERR_SHAPE;
    if (((static_cast<int64_t>(M) + 127) / 128) * ((w->N + 127) / 128) > (1 << 30)) return DH_ERR_SHAPE;
    if (!aligned(w->packed, 16) || !aligned(w->scale, 4) || !aligned(x, type_bytes(x_type)) ||
        !aligned(y, type_bytes(y_type)) || !aligned(error, 4))
        return DH_ERR_ALIGN;
    if (ws == nullptr) return DH_ERR_ARG;
    if (!aligned(ws, DH_WORKSPACE_ALIGN) || ws_bytes < dh::matmul_workspace_bytes(M, w->K)) return DH_ERR_WORKSPACE;
    a.packed = static_cast<const uint8_t*>(w->packed);
    a.g = w->scale;
    a.N = w->N;
    a.K = w->K;
    a.M = M;
    a.x = x;
    a.x_type = x_type;
    a.ldx = ldx;
    a.y = y;
    a.y_type = y_type;
    a.ldy = ldy;
    a.ws = ws;
    a.error = error;
    return DH_OK;
}

}  // namespace

extern "C" {

size_t nvfp4_matmul_packed_bytes(int N, int K) { return check_shape(N, K) == DH_OK ? dh::matmul_packed_bytes(N, K) : 0; }

size_t nvfp4_matmul_workspace_bytes(int M, int K) {
    return M < 1 || M > kMaxM || check_shape(64, K) != DH_OK ? 0 : dh::matmul_workspace_bytes(M, K);
}

int nvfp4_pack_matmul(const uint8_t* q, const uint8_t* sf, int N, int K, uint8_t* packed, void* stream) {
    if (q == nullptr || sf == nullptr || packed == nullptr) return DH_ERR_ARG;
    if (check_shape(N, K) != DH_OK) return DH_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(packed, 16)) return DH_ERR_ALIGN;
    return cuda_status(dh::launch_matmul_pack(q, sf, N, K, packed, static_cast<cudaStream_t>(stream)));
}

int nvfp4_matmul(const dh_matmul_t* w, const void* x, int x_type, int64_t ldx, int M, void* y, int y_type, int64_t ldy,
                 void* ws, size_t ws_bytes, unsigned int* error, void* stream) {
    dh::MatmulArgs a = {};
    const int st = check_matmul(w, x, x_type, ldx, M, y, y_type, ldy, ws, ws_bytes, error, a);
    return st != DH_OK ? st : cuda_status(dh::launch_matmul(a, static_cast<cudaStream_t>(stream)));
}

int nvfp4_matmul_wait_probe(const dh_matmul_t* w, const void* x, int M, void* y, void* ws, size_t ws_bytes, int role,
                            unsigned int rounds, unsigned int* error, void* stream) {
    if (w == nullptr || error == nullptr || role < 0 || role > 3 || rounds < 1 || rounds > 4096) return DH_ERR_ARG;
    dh::MatmulArgs a = {};
    const int st = check_matmul(w, x, DH_T_BF16, w->K, M, y, DH_T_BF16, w->N, ws, ws_bytes, error, a);
    if (st != DH_OK) return st;
    a.probe_role = role;
    a.probe_rounds = rounds;
    return cuda_status(dh::launch_matmul(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
