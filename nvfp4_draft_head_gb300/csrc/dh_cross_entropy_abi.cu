// C-ABI entry points of the vocabulary cross entropy: argument checks on the host, then the
// launches of dh_cross_entropy.cu. See include/drafthead.h.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/drafthead.h"
#include "dh_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? DH_OK : dh::record_cuda_error(e); }

// The library's own error word, laid out as the head of a workspace (dh::Workspace: the word comes
// first). In host code this name is a host-side stand-in: the address comes from
// cudaGetSymbolAddress.
static __device__ __align__(DH_WORKSPACE_ALIGN) unsigned int g_error_word;

constexpr int kMaxT = 1 << 24, kMaxN = 1 << 24, kMaxK = 1 << 20;

bool shape_ok(int T, int N, int K) {
    return T >= 1 && T <= kMaxT && N >= 1 && N <= kMaxN && K >= 8 && K <= kMaxK && K % 8 == 0 &&
           ((static_cast<int64_t>(T) + 255) / 256) * ((N + 255) / 256) <= (1 << 29) &&
           ((static_cast<int64_t>(T) + 255) / 256) * ((K + 255) / 256) <= (1 << 24) &&
           ((static_cast<int64_t>(N) + 255) / 256) * ((K + 255) / 256) <= (1 << 29);
}

// A [rows][K] matrix: 16-byte rows (their stride, below a tensor map's 2^40 bytes, means nothing
// for a single one).
int check_rows(const void* p, int64_t ld, int rows, int K) {
    if (rows > 1 && (ld < K || ld >= (1ll << 39))) return DH_ERR_SHAPE;
    return aligned(p, 16) && (rows == 1 || ld % 8 == 0) ? DH_OK : DH_ERR_ALIGN;
}

int64_t stride(int64_t ld, int rows, int K) { return rows > 1 ? ld : K; }

int check(const dh_cross_entropy_t* c, void* dhidden, int64_t ld_dhidden, void* dhead, int64_t ld_dhead, const void* ws,
          const unsigned int* error, dh::CrossEntropyArgs& a) {
    if (c == nullptr || c->hidden == nullptr || c->head == nullptr || c->tokens == nullptr || ws == nullptr) return DH_ERR_ARG;
    const int type = c->type & ~static_cast<int>(DH_CE_TWO_TERMS);
    if (type != DH_T_BF16 && type != DH_T_F16) return DH_ERR_ARG;
    if (dhidden == c->hidden || dhead == c->head || (dhidden != nullptr && dhidden == dhead)) return DH_ERR_ARG;   // not in place
    if (!shape_ok(c->T, c->N, c->K)) return DH_ERR_SHAPE;
    if (c->row_of != nullptr && c->V < 1) return DH_ERR_SHAPE;
    int st;
    if ((st = check_rows(c->hidden, c->ld_hidden, c->T, c->K)) != DH_OK) return st;
    if ((st = check_rows(c->head, c->ld_head, c->N, c->K)) != DH_OK) return st;
    if (dhidden != nullptr && (st = check_rows(dhidden, ld_dhidden, c->T, c->K)) != DH_OK) return st;
    if (dhead != nullptr && (st = check_rows(dhead, ld_dhead, c->N, c->K)) != DH_OK) return st;
    if (!aligned(c->tokens, 4) || !aligned(c->weight, 4) || !aligned(c->row_of, 4) || !aligned(error, 4)) return DH_ERR_ALIGN;
    a.hidden = c->hidden;
    a.head = c->head;
    a.type = type;
    a.two_terms = c->type != type;
    a.T = c->T;
    a.N = c->N;
    a.K = c->K;
    a.ld_hidden = stride(c->ld_hidden, c->T, c->K);
    a.ld_head = stride(c->ld_head, c->N, c->K);
    a.tokens = c->tokens;
    a.weight = c->weight;
    a.row_of = c->row_of;
    a.V = c->V;
    a.dhidden = dhidden;
    a.ld_dhidden = stride(ld_dhidden, c->T, c->K);
    a.dhead = dhead;
    a.ld_dhead = stride(ld_dhead, c->N, c->K);
    a.error = const_cast<unsigned int*>(error);
    return DH_OK;
}

int check_space(const dh::CrossEntropyArgs& a, void* ws, size_t ws_bytes) {
    return aligned(ws, DH_WORKSPACE_ALIGN) &&
                   ws_bytes >= dh::cross_entropy_workspace_bytes(a.T, a.N, a.K, a.loss != nullptr, a.dhidden != nullptr, a.dhead != nullptr,
                                                                  a.two_terms)
               ? DH_OK
               : DH_ERR_WORKSPACE;
}

}  // namespace

extern "C" {

size_t draft_head_cross_entropy_workspace_bytes(int T, int N, int K, unsigned int outputs) {
    const unsigned int what = outputs & ~DH_CE_TWO_TERMS;
    if (!shape_ok(T, N, K) || (what & ~7u) != 0u || what == 0u) return 0;
    return dh::cross_entropy_workspace_bytes(T, N, K, (what & DH_CE_LOSS) != 0, (what & DH_CE_DHIDDEN) != 0, (what & DH_CE_DHEAD) != 0,
                                             what != outputs);
}

int draft_head_cross_entropy(const dh_cross_entropy_t* c, float* loss, float* lse, float* rest, void* dhidden, int64_t ld_dhidden,
                             void* dhead, int64_t ld_dhead, void* ws, size_t ws_bytes, unsigned int* error, void* stream) {
    if (loss == nullptr) return DH_ERR_ARG;
    dh::CrossEntropyArgs a = {};
    int st = check(c, dhidden, ld_dhidden, dhead, ld_dhead, ws, error, a);
    if (st != DH_OK) return st;
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(rest, 4)) return DH_ERR_ALIGN;
    a.loss = loss;
    a.lse = lse;
    a.rest = rest;
    if ((st = check_space(a, ws, ws_bytes)) != DH_OK) return st;
    a.ws = ws;
    return cuda_status(dh::launch_cross_entropy(a, static_cast<cudaStream_t>(stream)));
}

int draft_head_cross_entropy_backward(const dh_cross_entropy_t* c, const float* lse, const float* rest, void* dhidden,
                                      int64_t ld_dhidden, void* dhead, int64_t ld_dhead, void* ws, size_t ws_bytes,
                                      unsigned int* error, void* stream) {
    if (lse == nullptr || (dhidden == nullptr && dhead == nullptr)) return DH_ERR_ARG;
    dh::CrossEntropyArgs a = {};
    int st = check(c, dhidden, ld_dhidden, dhead, ld_dhead, ws, error, a);
    if (st != DH_OK) return st;
    if (!aligned(lse, 4) || !aligned(rest, 4)) return DH_ERR_ALIGN;
    a.lse_in = lse;
    a.rest_in = rest;
    if ((st = check_space(a, ws, ws_bytes)) != DH_OK) return st;
    a.ws = ws;
    return cuda_status(dh::launch_cross_entropy(a, static_cast<cudaStream_t>(stream)));
}

int draft_head_cross_entropy_error_word(void** word) {
    if (word == nullptr) return DH_ERR_ARG;
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, g_error_word);
    if (e != cudaSuccess) return dh::record_cuda_error(e);
    *word = p;
    return DH_OK;
}

int draft_head_cross_entropy_wait_probe(const dh_cross_entropy_t* c, float* loss, void* ws, size_t ws_bytes, int role, unsigned int rounds,
                                        unsigned int* error, void* stream) {
    if (loss == nullptr || error == nullptr || role < 0 || role > 2 || rounds < 1 || rounds > 4096) return DH_ERR_ARG;
    dh::CrossEntropyArgs a = {};
    int st = check(c, nullptr, 0, nullptr, 0, ws, error, a);
    if (st != DH_OK) return st;
    if (!aligned(loss, 4)) return DH_ERR_ALIGN;
    a.loss = loss;
    if ((st = check_space(a, ws, ws_bytes)) != DH_OK) return st;
    a.ws = ws;
    a.probe_role = role;
    a.probe_rounds = rounds;
    return cuda_status(dh::launch_cross_entropy(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
