// C ABI of the paged step (plan, trees, cache append, attention over the paged
// cache, sampling): argument checking and launch configuration. Declarations and the
// contract of every entry point are in include/moe_decode.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "moe_decode.h"
#include "host.h"
#include "layer_params.h"
#include "paged.h"
#include "paged_host.h"

namespace {

using moe::DeviceInfo;
using moe::EncodeTiled;
using moe::aligned16;
using moe::aligned4;
using moe::aligned8;
using moe::check_cache;
using moe::check_ws;
using moe::device_info;
using moe::encode_tiled;
using moe::g_last_launches;
using moe::g_opt;
using moe::launched;
using moe::stride_ok;

static_assert(moe::kMaxRequests == MOE_PAGED_MAX_REQUESTS, "request limit");
static_assert(moe::kSampleMaxSlice * 16 == MOE_SAMPLE_MAX_VOCAB, "vocabulary limit");
static_assert(moe::kAttnMaxGrid == MOE_MAX_GRID, "grid limit");
static_assert(moe::kTreeTokens == MOE_TREE_MAX_TOKENS, "tokens of a tree");
static_assert(moe::kCtlBytes <= MOE_PAGED_WORKSPACE_BYTES, "control block");

// Tensor map of a cache: (64 dimensions, token of the block, which 64, head,
// block), boxes of `panels` times 64 dimensions by `box` tokens in the 128-byte
// swizzle.
bool cache_map(CUtensorMap* m, const moe_kv_cache* c, void* base, int64_t bs, int64_t ts, int64_t hs, int box,
               int panels) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[5] = {64, (cuuint64_t)c->block_size, (cuuint64_t)(c->head_dim / 64), (cuuint64_t)c->kv_heads,
                                (cuuint64_t)c->n_blocks};
    const cuuint64_t strides[4] = {(cuuint64_t)ts * 2, 128, (cuuint64_t)hs * 2, (cuuint64_t)bs * 2};
    const cuuint32_t boxes[5] = {64, (cuuint32_t)box, (cuuint32_t)panels, 1, 1}, steps[5] = {1, 1, 1, 1, 1};
    return enc(m, c->dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, base, dims,
               strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Attention over a 16-bit cache; masks: of trees, null for none.
int attend(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads, const moe_kv_cache* cache,
           const int32_t* block_tables, int max_blocks, const int32_t* q_start, const int32_t* seq_lens, int B, float scale,
           int window, const uint64_t* masks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > 32) return MOE_ESHAPE;
    const int group = q_heads / cache->kv_heads;
    if (T < 0 || (int64_t)T * group >= (1 << 28)) return MOE_ESHAPE;
    if (B < 1 || B > MOE_PAGED_MAX_REQUESTS || max_blocks < 1 || window < 0) return MOE_ESHAPE;
    if (!(scale == scale) || std::isinf(scale)) return MOE_EINVAL;
    if (!block_tables || !q_start || !seq_lens) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!q || !out) return MOE_EINVAL;
    if (!stride_ok(q_token_stride, 0) || !stride_ok(q_head_stride, 0)) return MOE_ESHAPE;
    if (!aligned16(q) || !aligned16(out) || !aligned4(lse) || !aligned4(block_tables) || !aligned4(q_start) ||
        !aligned4(seq_lens))
        return MOE_EALIGN;
    rc = check_ws(ws, ws_bytes, moe_paged_attention_workspace_bytes(q_heads, cache));
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::AttnParams p = {};
    p.G = g_opt.grid_ctas > 0 ? g_opt.grid_ctas : std::min(dev.sms, MOE_MAX_GRID);
    if (p.G > dev.sms || p.G > MOE_MAX_GRID) return MOE_EINVAL;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.tables = block_tables;
    p.q_start = q_start;
    p.seq = seq_lens;
    p.ctrl = static_cast<unsigned*>(ws);
    p.arrived = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(ws) + MOE_PAGED_WORKSPACE_BYTES);
    p.part = reinterpret_cast<float*>(p.arrived + 3 * MOE_MAX_GRID);
    p.chunk_part = p.part + (size_t)MOE_MAX_GRID * 2 * moe::attn_part_floats(moe::kAttnRows, cache->head_dim);
    p.q_token = q_token_stride;
    p.q_head = q_head_stride;
    p.T = T;
    p.B = B;
    p.heads = q_heads;
    p.kv_heads = cache->kv_heads;
    p.group = group;
    p.group_magic = ((1ull << 36) + group - 1) / group;
    p.max_blocks = max_blocks;
    p.block_size = cache->block_size;
    p.n_blocks = cache->n_blocks;
    // copies of the largest power of two that divides the block: none ends
    // beyond a block, and a tile is a whole number of them
    p.box_shift = std::min(__builtin_ctz((unsigned)cache->block_size), 7);
    p.box = 1 << p.box_shift;
    p.window = window;
    p.scale_log2 = (scale > 0.f ? scale : 1.f / std::sqrt((float)cache->head_dim)) * 1.44269504088896341f;
    p.timeout_ns = (unsigned long long)g_opt.timeout_ns;
    p.hold_back = g_opt.hold_back ? 1 : 0;
    p.tree = reinterpret_cast<const unsigned long long*>(masks);
    CUtensorMap maps[4];
    for (int i = 0; i < (moe::attn_may_chunk(p) ? 4 : 2); ++i) {
        const int panels = i < 2 ? cache->head_dim / 64 : 1;
        const bool ok = i % 2 == 0 ? cache_map(&maps[i], cache, cache->k, cache->k_block_stride, cache->k_token_stride,
                                               cache->k_head_stride, p.box, panels)
                                   : cache_map(&maps[i], cache, cache->v, cache->v_block_stride, cache->v_token_stride,
                                               cache->v_head_stride, p.box, panels);
        if (!ok) return MOE_ECUDA;
    }
    int n = 0;
    const cudaError_t e = moe::launch_attn(p, maps, cache->head_dim, cache->dtype, static_cast<cudaStream_t>(stream), &n);
    return launched(e, n);
}

}  // namespace

extern "C" {

int moe_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, const int32_t* free_list, int n_free,
                   const int32_t* free_head, int32_t* block_tables, int max_blocks, int block_size,
                   int32_t* q_start, int32_t* seq_lens, int32_t* slot_map, int32_t* positions, int T,
                   int32_t* taken, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    if (B < 1 || B > MOE_PAGED_MAX_REQUESTS || n_free < 0 || max_blocks < 1 || block_size < 1 || T < 0)
        return MOE_ESHAPE;
    if (!ctx_lens || !new_lens || (n_free > 0 && !free_list) || !block_tables || !q_start || !seq_lens ||
        (T > 0 && !slot_map) || !taken)
        return MOE_EINVAL;
    // no input may be overwritten while another CTA reads it
    for (const void* o : {(const void*)q_start, (const void*)seq_lens, (const void*)slot_map, (const void*)positions,
                          (const void*)taken, (const void*)block_tables})
        if (o && (o == ctx_lens || o == new_lens || o == free_list || o == free_head)) return MOE_EINVAL;
    for (const void* a : {(const void*)ctx_lens, (const void*)new_lens, (const void*)free_list,
                          (const void*)free_head, (const void*)block_tables, (const void*)q_start,
                          (const void*)seq_lens, (const void*)slot_map, (const void*)positions, (const void*)taken})
        if (!aligned4(a)) return MOE_EALIGN;
    int rc = check_ws(ws, ws_bytes, MOE_PAGED_WORKSPACE_BYTES);
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::PlanParams p = {};
    p.ctx = ctx_lens;
    p.fresh = new_lens;
    p.free_list = free_list;
    p.free_head = free_head;
    p.tables = block_tables;
    p.q_start = q_start;
    p.seq = seq_lens;
    p.slots = slot_map;
    p.positions = positions;
    p.taken = taken;
    p.ctrl = static_cast<unsigned*>(ws);
    p.B = B;
    p.n_free = n_free;
    p.max_blocks = max_blocks;
    p.block_size = block_size;
    p.T = T;
    return launched(moe::launch_paged_plan(p, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

int moe_paged_append(const void* k_new, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                     int64_t v_token_stride, int64_t v_head_stride, int T, const int32_t* slot_map,
                     const moe_kv_cache* cache, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    int rc = check_cache(cache);
    if (rc) return rc;
    if (T < 0) return MOE_ESHAPE;
    if (T == 0) return MOE_OK;
    if (!k_new || !v_new || !slot_map) return MOE_EINVAL;
    if (!stride_ok(k_token_stride, 0) || !stride_ok(k_head_stride, 0) || !stride_ok(v_token_stride, 0) ||
        !stride_ok(v_head_stride, 0))
        return MOE_ESHAPE;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(slot_map)) return MOE_EALIGN;
    rc = check_ws(ws, ws_bytes, MOE_PAGED_WORKSPACE_BYTES);
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::AppendParams p = {};
    p.src[0] = static_cast<const uint16_t*>(k_new);
    p.src[1] = static_cast<const uint16_t*>(v_new);
    p.src_token[0] = k_token_stride;
    p.src_token[1] = v_token_stride;
    p.src_head[0] = k_head_stride;
    p.src_head[1] = v_head_stride;
    p.dst[0] = static_cast<uint16_t*>(cache->k);
    p.dst[1] = static_cast<uint16_t*>(cache->v);
    p.dst_block[0] = cache->k_block_stride;
    p.dst_block[1] = cache->v_block_stride;
    p.dst_token[0] = cache->k_token_stride;
    p.dst_token[1] = cache->v_token_stride;
    p.dst_head[0] = cache->k_head_stride;
    p.dst_head[1] = cache->v_head_stride;
    p.slots = slot_map;
    p.ctrl = static_cast<unsigned*>(ws);
    p.T = T;
    p.heads = cache->kv_heads;
    p.dim_shift = cache->head_dim == 64 ? 3 : 4;
    p.block_size = cache->block_size;
    p.n_slots = (int64_t)cache->n_blocks * cache->block_size;
    return launched(moe::launch_paged_append(p, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

size_t moe_paged_attention_workspace_bytes(int q_heads, const moe_kv_cache* cache) {
    if (check_cache(cache) != MOE_OK) return 0;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > 32) return 0;
    return MOE_PAGED_WORKSPACE_BYTES + 3 * MOE_MAX_GRID * sizeof(unsigned) +
           (size_t)MOE_MAX_GRID * 2 * moe::attn_part_floats(moe::kAttnRows + moe::kAttnChunkRows, cache->head_dim) *
               sizeof(float);
}

int moe_paged_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads,
                        const moe_kv_cache* cache, const int32_t* block_tables, int max_blocks,
                        const int32_t* q_start, const int32_t* seq_lens, int B, float scale, int window, void* out,
                        float* lse, void* ws, size_t ws_bytes, void* stream) {
    return attend(q, q_token_stride, q_head_stride, T, q_heads, cache, block_tables, max_blocks, q_start, seq_lens, B, scale,
                  window, nullptr, out, lse, ws, ws_bytes, stream);
}

int moe_paged_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads,
                             const moe_kv_cache* cache, const int32_t* block_tables, int max_blocks,
                             const int32_t* q_start, const int32_t* seq_lens, const uint64_t* masks, int B, float scale,
                             void* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    if (!masks) return MOE_EINVAL;
    if (!aligned8(masks)) return MOE_EALIGN;
    return attend(q, q_token_stride, q_head_stride, T, q_heads, cache, block_tables, max_blocks, q_start, seq_lens, B, scale, 0,
                  masks, out, lse, ws, ws_bytes, stream);
}

int moe_tree_plan(const int32_t* parents, const int32_t* q_start, const int32_t* seq_lens, int B, int T, uint64_t* masks,
                  int32_t* positions, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    if (B < 1 || B > MOE_PAGED_MAX_REQUESTS || T < 0) return MOE_ESHAPE;
    if (T == 0) return MOE_OK;
    if (!parents || !q_start || !seq_lens || !masks) return MOE_EINVAL;
    // no input may be overwritten while another CTA reads it
    for (const void* o : {(const void*)masks, (const void*)positions})
        if (o && (o == parents || o == q_start || o == seq_lens)) return MOE_EINVAL;
    for (const void* a : {(const void*)parents, (const void*)q_start, (const void*)seq_lens, (const void*)positions})
        if (!aligned4(a)) return MOE_EALIGN;
    if (!aligned8(masks)) return MOE_EALIGN;
    int rc = check_ws(ws, ws_bytes, MOE_PAGED_WORKSPACE_BYTES);
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::TreeParams p = {};
    p.parents = parents;
    p.q_start = q_start;
    p.seq = seq_lens;
    p.masks = reinterpret_cast<unsigned long long*>(masks);
    p.positions = positions;
    p.ctrl = static_cast<unsigned*>(ws);
    p.B = B;
    p.T = T;
    return launched(moe::launch_tree_plan(p, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

int moe_sample(const void* logits, int dtype, int M, int V, int64_t row_stride, const float* u,
               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
               int32_t* token, float* prob, void* stream) {
    g_last_launches = 0;
    if (dtype != 0 && dtype != 1) return MOE_ESHAPE;
    if (M < 1 || V < 1 || V > MOE_SAMPLE_MAX_VOCAB || row_stride < V) return MOE_ESHAPE;
    if (!logits || !u || !token) return MOE_EINVAL;
    if ((reinterpret_cast<uintptr_t>(logits) & (dtype == 0 ? 3u : 1u)) != 0) return MOE_EALIGN;
    for (const void* a : {(const void*)u, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                          (const void*)min_p, (const void*)token, (const void*)prob})
        if (!aligned4(a)) return MOE_EALIGN;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc) return rc;
    moe::SampleParams p = {};
    p.logits = logits;
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.token = token;
    p.prob = prob;
    p.row_stride = row_stride;
    p.V = V;
    return launched(moe::launch_sample(p, M, dtype, static_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
