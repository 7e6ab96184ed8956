// Launch parameters of the paged-step kernels (plan, cache append, attention
// over the paged cache, sampling). Plain C++, shared by the host launchers
// and the kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace moe {

constexpr int kMaxRequests = 4096;

struct PlanParams {
    const int32_t* ctx;
    const int32_t* fresh;  // new tokens of each request
    const int32_t* free_list;
    const int32_t* free_head;  // may be null
    int32_t* tables;
    int32_t* q_start;
    int32_t* seq;
    int32_t* slots;
    int32_t* positions;  // may be null
    int32_t* taken;
    unsigned* ctrl;
    int B, n_free, max_blocks, block_size, T;
};

struct TreeParams {
    const int32_t* parents;
    const int32_t* q_start;
    const int32_t* seq;
    unsigned long long* masks;
    int32_t* positions;  // may be null
    unsigned* ctrl;
    int B, T;
};

struct AppendParams {
    const uint16_t* src[2];  // new keys, new values
    uint16_t* dst[2];        // the cache's K and V
    int64_t src_token[2], src_head[2];
    int64_t dst_block[2], dst_token[2], dst_head[2];
    const int32_t* slots;
    unsigned* ctrl;
    int T, heads, dim_shift;  // head_dim = 8 << dim_shift
    int block_size;
    int64_t n_slots;
};

// Rotation of queries and keys, and the write of keys and values, by token
// (rope.cu). Sources and destinations: 0 queries, 1 keys, 2 values.
struct RotateParams {
    const uint16_t* src[3];
    int64_t src_token[3], src_head[3];
    uint16_t* dst[2];  // rotated queries and (without a cache) keys
    int64_t dst_token[2], dst_head[2];
    int heads[3];
    const int32_t* positions;         // null: no rotation
    const unsigned long long* turns;  // of a pair's frequency, in 2^-64
    float scale;
    int rotary_dim, interleaved;
    int T, head_dim;
    int lanes, per;  // lanes of a head (16 elements each), heads that a warp takes at a time
    int split;       // warps that share a token
    // the cache that keys and values go to
    const int32_t* slots;
    uint8_t* cache[2];
    uint8_t* cache_scale[2];  // e4m3 codes alone
    int64_t cache_block[2], cache_token[2], cache_head[2];  // bytes
    int block_size;
    int64_t n_slots;
    unsigned* ctrl;
};
// Where keys go.
enum { kRotateRows = 0, kRotateCache16 = 1, kRotateCache8 = 2 };
cudaError_t launch_rotate(RotateParams p, int to, int dtype, int sms, cudaStream_t stream);

// Slots of a cache back into rows.
struct ReadParams {
    const uint8_t* cache[2];
    const uint8_t* cache_scale[2];
    int64_t cache_block[2], cache_token[2], cache_head[2];  // bytes
    uint16_t* dst[2];
    int64_t dst_token[2], dst_head[2];
    const int32_t* slots;
    unsigned* ctrl;
    int T, heads, lane_shift;  // head_dim = 16 << lane_shift
    int block_size, split;
    int64_t n_slots;
};
// from: 0 a cache of 16 bits, 1 of e4m3 codes
cudaError_t launch_read(ReadParams p, int from, int dtype, int sms, cudaStream_t stream);

constexpr int kSampleThreads = 512;
constexpr int kSampleMaxSlice = 45056;  // logits of a row that one CTA holds

struct SampleParams {
    const void* logits;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;
    float* prob;
    int64_t row_stride;
    int V, C, slice;
};

// Attention over the paged cache. Keys are taken in tiles of kAttnTile.
constexpr int kAttnTile = 128;
constexpr int kAttnRows = 32;       // query rows of an item of the decode kernel
constexpr int kAttnChunkRows = 256; // and of the chunk kernel
// Requests with more query rows a kv head than this go to the chunk kernel.
constexpr int kAttnFewRows = 64;
constexpr int kAttnMaxGrid = 256;   // CTAs of a launch (workspace sizing)

struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    float* lse;  // may be null
    const int32_t* tables;
    const int32_t* q_start;
    const int32_t* seq;
    unsigned* ctrl;
    float* part;        // partial results of items that span CTAs, [G][2]
    float* chunk_part;  // and those of the chunk kernel's
    // parts that are in place of the item that spans from CTA c, [3][kAttnMaxGrid]:
    // of the decode kernel, of the chunk kernel's two slots. Zero between calls.
    unsigned* arrived;
    int64_t q_token, q_head;
    int T, B, heads, kv_heads, group;
    unsigned long long group_magic;  // ceil(2^36 / group): x / group = x * magic >> 36 for x < 2^28
    int max_blocks, block_size, n_blocks;
    int box, box_shift;  // keys that one copy brings, as a power of two
    int window;
    int G;       // CTAs
    float scale_log2;  // scale * log2(e)
    unsigned long long timeout_ns;
    int hold_back;  // test hook: 1, a CTA's first keys (scores, in the chunk kernel) never come
    // Trees of drafted tokens (null: none): of each token row the new tokens of
    // its request that it sees, where the request has at most kTreeTokens.
    const unsigned long long* tree;
    const uint8_t* scales[2];  // of K and V of a cache of 8-bit values
};
constexpr int kTreeTokens = 64;

// Whether any request of the call may have many rows.
inline bool attn_may_chunk(const AttnParams& p) { return (int64_t)p.T * p.group > kAttnFewRows; }
// The decode kernel and the chunk kernel (where any request may have many
// rows). maps: CUtensorMaps of K and V whose boxes hold all
// dimensions of `box` keys, then of K and V in boxes of 64 dimensions (for the
// chunk kernel alone).
cudaError_t launch_attn(const AttnParams& p, const void* maps, int head_dim, int dtype, cudaStream_t stream,
                        int* launches);
cudaError_t launch_attn_chunk(const AttnParams& p, const void* k_map, const void* v_map, int head_dim, int dtype,
                              cudaStream_t stream);
// Over a cache of 8-bit values: maps of K and V whose boxes hold all dimensions
// of `box` keys.
cudaError_t launch_attn_codes(const AttnParams& p, const void* k_map, const void* v_map, int head_dim, int dtype,
                              cudaStream_t stream);
// Floats of one partial result of `rows` rows.
constexpr int attn_part_floats(int rows, int head_dim) { return rows * (head_dim + 2); }

cudaError_t launch_paged_plan(const PlanParams& p, int sms, cudaStream_t stream);
cudaError_t launch_tree_plan(const TreeParams& p, int sms, cudaStream_t stream);
cudaError_t launch_paged_append(const AppendParams& p, int sms, cudaStream_t stream);
// Chooses p.C and p.slice.
cudaError_t launch_sample(SampleParams p, int M, int dtype, cudaStream_t stream);

}  // namespace moe
