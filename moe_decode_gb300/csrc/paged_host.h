// Checks and helpers that the paged step's entry points share (api_paged.cu,
// api_paged8.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "host.h"
#include "moe_decode.h"

namespace moe {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

inline int check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws) return MOE_EWORKSPACE;
    if (!aligned16(ws)) return MOE_EALIGN;
    return ws_bytes < need ? MOE_EWORKSPACE : MOE_OK;
}

inline bool stride_ok(int64_t s, int least) { return s >= least && s % 8 == 0 && s < (1LL << 36); }

inline int check_cache(const moe_kv_cache* c) {
    if (!c || !c->k || !c->v) return MOE_EINVAL;
    if (c->dtype != 0 && c->dtype != 1) return MOE_ESHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return MOE_ESHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 256) return MOE_ESHAPE;
    if (c->block_size < 8 || c->block_size > 1024 || c->block_size % 8 != 0) return MOE_ESHAPE;
    if (c->n_blocks < 1 || (int64_t)c->n_blocks * c->block_size > 0x7fffffffLL) return MOE_ESHAPE;
    for (int64_t s : {c->k_block_stride, c->k_token_stride, c->k_head_stride, c->v_block_stride, c->v_token_stride,
                      c->v_head_stride})
        if (!stride_ok(s, c->head_dim)) return MOE_ESHAPE;
    if (!aligned16(c->k) || !aligned16(c->v)) return MOE_EALIGN;
    return MOE_OK;
}

inline int check_cache8(const moe_kv_cache8* c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return MOE_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128) return MOE_ESHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 256) return MOE_ESHAPE;
    if (c->block_size < 16 || c->block_size > 1024 || c->block_size % 16 != 0) return MOE_ESHAPE;
    if (c->n_blocks < 1 || (int64_t)c->n_blocks * c->block_size > 0x7fffffffLL) return MOE_ESHAPE;
    for (int64_t s : {c->k_block_stride, c->k_token_stride, c->k_head_stride, c->v_block_stride, c->v_token_stride,
                      c->v_head_stride})
        if (!stride_ok(s, c->head_dim) || s % 16 != 0) return MOE_ESHAPE;
    for (const void* a : {(const void*)c->k, (const void*)c->v, (const void*)c->k_scale, (const void*)c->v_scale})
        if (!aligned16(a)) return MOE_EALIGN;
    return MOE_OK;
}

inline int launched(cudaError_t e, int n) {
    g_last_launches = n;
    if (e == cudaSuccess) return MOE_OK;
    cudaGetLastError();
    return MOE_ECUDA;
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// The driver's tensor-map encoder, looked up once (the library links the
// runtime alone).
inline EncodeTiled encode_tiled() {
    static EncodeTiled f = [] {
        void* sym = nullptr;
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &sym, 12000, cudaEnableDefault, &res) !=
                cudaSuccess ||
            res != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            sym = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(sym);
    }();
    return f;
}

}  // namespace moe
