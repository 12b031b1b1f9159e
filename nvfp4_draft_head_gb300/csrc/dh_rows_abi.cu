// C-ABI entry points of the operators on logits rows: argument checks on the
// host, then the launches of dh_logprobs.cu and dh_distill.cu. See
// include/drafthead.h.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/drafthead.h"
#include "dh_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? DH_OK : dh::record_cuda_error(e); }

// Bytes of an element type, 0 for an unknown one.
int type_bytes(int type) { return type == DH_T_BF16 || type == DH_T_F16 ? 2 : type == DH_T_F32 ? 4 : 0; }

constexpr int kMaxRows = 1 << 27;   // rows times CTAs per row fit a grid

int check_logits(const dh_logits_t* lg) {
    if (lg == nullptr || lg->z == nullptr) return DH_ERR_ARG;
    const int b = type_bytes(lg->type);
    if (b == 0) return DH_ERR_ARG;
    // the kernels scale exponents by (1 / t) log2(e), which is infinite for the smallest t
    if (!(lg->temperature > 0.0f) || !std::isfinite(lg->temperature) || !std::isfinite(1.0f / lg->temperature * 1.44269504f))
        return DH_ERR_ARG;
    if (lg->M < 1 || lg->M > kMaxRows || lg->C < 1 || lg->C > (1 << 30)) return DH_ERR_SHAPE;
    if (lg->M > 1 && lg->ld < lg->C) return DH_ERR_SHAPE;
    if (lg->row_of != nullptr && lg->V < 1) return DH_ERR_SHAPE;
    if (!aligned(lg->z, b) || !aligned(lg->row_of, 4) || !aligned(lg->idx, 4)) return DH_ERR_ALIGN;
    return DH_OK;
}

int check_teacher(const int32_t* ids, const void* val, int val_type, int K) {
    if (ids == nullptr || val == nullptr || type_bytes(val_type) == 0) return DH_ERR_ARG;
    if (K < 1 || K > DH_MAX_TEACHER) return DH_ERR_SHAPE;
    if (!aligned(ids, 4) || !aligned(val, type_bytes(val_type))) return DH_ERR_ALIGN;
    return DH_OK;
}

int check_gradient(const dh_logits_t* lg, const void* dz, int64_t ld_dz) {
    if (lg->M > 1 && ld_dz < lg->C) return DH_ERR_SHAPE;
    if (dz == lg->z && lg->M > 1 && ld_dz != lg->ld) return DH_ERR_SHAPE;   // in place: the same layout
    return aligned(dz, type_bytes(lg->type)) ? DH_OK : DH_ERR_ALIGN;
}

dh::DistillArgs distill_args(const dh_logits_t* lg, const int32_t* ids, const void* val, int val_type, int K,
                              const float* weight) {
    dh::DistillArgs a = {};
    a.z = lg->z;
    a.ld = lg->ld;
    a.M = lg->M;
    a.C = lg->C;
    a.t = lg->temperature;
    a.inv_t = 1.0f / lg->temperature;
    a.row_of = lg->row_of;
    a.V = lg->V;
    a.ids = ids;
    a.val = val;
    a.val_type = val_type;
    a.K = K;
    a.weight = weight;
    return a;
}

}  // namespace

extern "C" {

int draft_head_row_map(const int32_t* idx, int n_kept, int32_t* row_of, int V, void* stream) {
    if (idx == nullptr || row_of == nullptr) return DH_ERR_ARG;
    if (n_kept < 1 || V < 1) return DH_ERR_SHAPE;
    if (!aligned(idx, 4) || !aligned(row_of, 4)) return DH_ERR_ALIGN;
    return cuda_status(dh::launch_row_map(idx, n_kept, row_of, V, static_cast<cudaStream_t>(stream)));
}

int draft_head_token_logprobs(const dh_logits_t* lg, const int32_t* tokens, int G, float* logp, float* entropy, float* lse,
                              int top_k, float* top_logp, int32_t* top_ids, void* stream) {
    const int st = check_logits(lg);
    if (st != DH_OK) return st;
    if (G < 0 || top_k < 0 || top_k > DH_MAX_TOP) return DH_ERR_SHAPE;
    if (G > 0 && (tokens == nullptr || logp == nullptr)) return DH_ERR_ARG;
    if (top_k > 0 && (top_logp == nullptr || top_ids == nullptr)) return DH_ERR_ARG;
    for (const void* p : {static_cast<const void*>(tokens), static_cast<const void*>(logp), static_cast<const void*>(entropy),
                          static_cast<const void*>(lse), static_cast<const void*>(top_logp), static_cast<const void*>(top_ids)})
        if (!aligned(p, 4)) return DH_ERR_ALIGN;
    dh::LogprobArgs a = {};
    a.z = lg->z;
    a.ld = lg->ld;
    a.M = lg->M;
    a.C = lg->C;
    a.inv_t = 1.0f / lg->temperature;
    a.row_of = lg->row_of;
    a.V = lg->V;
    a.idx = lg->idx;
    a.tokens = tokens;
    a.G = G;
    a.logp = logp;
    a.entropy = entropy;
    a.lse = lse;
    a.k = top_k;
    a.top_logp = top_logp;
    a.top_ids = top_ids;
    return cuda_status(dh::launch_token_logprobs(a, lg->type, static_cast<cudaStream_t>(stream)));
}

int draft_head_distill(const dh_logits_t* lg, const int32_t* ids, const void* val, int val_type, int K, const float* weight,
                       float* loss, float* lse, void* dz, int64_t ld_dz, void* stream) {
    int st = check_logits(lg);
    if (st != DH_OK) return st;
    if ((st = check_teacher(ids, val, val_type, K)) != DH_OK) return st;
    if (loss == nullptr || (lse != nullptr && dz != nullptr)) return DH_ERR_ARG;
    if (!aligned(weight, 4) || !aligned(loss, 4) || !aligned(lse, 4)) return DH_ERR_ALIGN;
    if (dz != nullptr && (st = check_gradient(lg, dz, ld_dz)) != DH_OK) return st;
    dh::DistillArgs a = distill_args(lg, ids, val, val_type, K, weight);
    a.loss = loss;
    a.lse = lse;
    a.dz = dz;
    a.ld_dz = ld_dz;
    return cuda_status(dh::launch_distill(a, lg->type, dz != nullptr ? dh::kDistillBoth : dh::kDistillForward,
                                          static_cast<cudaStream_t>(stream)));
}

int draft_head_distill_backward(const dh_logits_t* lg, const int32_t* ids, const void* val, int val_type, int K,
                                const float* lse, const float* weight, void* dz, int64_t ld_dz, void* stream) {
    int st = check_logits(lg);
    if (st != DH_OK) return st;
    if ((st = check_teacher(ids, val, val_type, K)) != DH_OK) return st;
    if (lse == nullptr || dz == nullptr) return DH_ERR_ARG;
    if (!aligned(weight, 4) || !aligned(lse, 4)) return DH_ERR_ALIGN;
    if ((st = check_gradient(lg, dz, ld_dz)) != DH_OK) return st;
    dh::DistillArgs a = distill_args(lg, ids, val, val_type, K, weight);
    a.lse_in = lse;
    a.dz = dz;
    a.ld_dz = ld_dz;
    return cuda_status(dh::launch_distill(a, lg->type, dh::kDistillBackward, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
