// C ABI of rotary positions, of the paged cache of 8-bit values (write, reading
// back, attention) and of reading slots back: argument checking and launch configuration. Declarations and the
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
using moe::aligned16;
using moe::aligned4;
using moe::aligned8;
using moe::check_cache;
using moe::check_cache8;
using moe::check_ws;
using moe::device_info;
using moe::encode_tiled;
using moe::g_last_launches;
using moe::g_opt;
using moe::launched;
using moe::stride_ok;

constexpr double kTwoPi = 6.283185307179586476925286766559, kTwoPiLo = 2.4492935982947064e-16;  // and what it lacks

// The part of a turn that a position adds, in 2^-64 of one. (By a division of 64
// bits, so that pi in 64 bits is half a turn.)
uint64_t turns_of(double radians) {
    double t = radians / kTwoPi;
    t -= std::floor(t);
    const double units = std::nearbyint(std::ldexp(t, 64));
    return units >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(units);
}

// A number as the sum of two of 64 bits, some 106 bits of it: a table's turns are
// good to their last unit, 2^-64, and a position multiplies what they are off by.
// (Sums and products without error by two-sum and by a fused multiply-add.)
struct Wide {
    double hi, lo;
    Wide(double h, double l = 0) : hi(h), lo(l) {}
};
Wide sum_of(double a, double b) {
    const double s = a + b, c = s - a;
    return Wide(s, (a - (s - c)) + (b - c));
}
Wide operator+(Wide a, Wide b) {
    const Wide s = sum_of(a.hi, b.hi), t = sum_of(a.lo, b.lo), u = sum_of(s.hi, s.lo + t.hi);
    return sum_of(u.hi, u.lo + t.lo);
}
Wide operator-(Wide a) { return Wide(-a.hi, -a.lo); }
Wide operator*(Wide a, Wide b) {
    const double p = a.hi * b.hi;
    return sum_of(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
Wide operator/(Wide a, Wide b) {
    const double q = a.hi / b.hi;
    return sum_of(q, (a + -(b * q)).hi / b.hi);
}
// x with x^n = a (a > 0): one of Newton's steps from 64 bits.
Wide root_of(Wide a, int n) {
    const double x = std::pow(a.hi, 1.0 / n);
    Wide power = 1, square = x;
    for (int i = n; i > 0; i >>= 1) {
        if (i & 1) power = power * square;
        square = square * square;
    }
    if (!std::isfinite(power.hi)) return x;  // (next to the largest number of 64 bits)
    return sum_of(x, x * (((a + -power) / power).hi / n));
}
// A frequency over 2 pi, its whole part dropped, in 2^-64.
uint64_t turns_of(Wide radians) {
    const Wide t = radians / Wide(kTwoPi, kTwoPiLo);
    const Wide f = sum_of(t.hi - std::floor(t.hi), t.lo - std::nearbyint(t.lo));  // (between -1 and 2)
    const double half = std::ldexp(f.hi, 32), whole = std::floor(half);
    return (static_cast<uint64_t>(static_cast<int64_t>(whole)) << 32) +
           static_cast<uint64_t>(static_cast<int64_t>(std::nearbyint(std::ldexp(half - whole, 32) + std::ldexp(f.lo, 64))));
}

int check_angles(const moe_rope_angles* a, int head_dim) {
    if (!a || !a->turns) return MOE_EINVAL;
    if (a->rotary_dim < 16 || a->rotary_dim % 16 != 0 || a->rotary_dim > head_dim) return MOE_ESHAPE;
    if (a->interleaved != 0 && a->interleaved != 1) return MOE_EINVAL;
    if (!std::isfinite(a->scale)) return MOE_EINVAL;
    return aligned8(a->turns) ? MOE_OK : MOE_EALIGN;
}

struct Rows {
    const void* p;
    int64_t token, head;
};
int check_rows(const Rows& in) {
    if (!in.p) return MOE_EINVAL;
    if (!stride_ok(in.token, 0) || !stride_ok(in.head, 0)) return MOE_ESHAPE;
    return aligned16(in.p) ? MOE_OK : MOE_EALIGN;
}
int check_out(const Rows& out, int head_dim) {
    if (!out.p) return MOE_EINVAL;
    if (!stride_ok(out.token, head_dim) || !stride_ok(out.head, head_dim)) return MOE_ESHAPE;
    return aligned16(out.p) ? MOE_OK : MOE_EALIGN;
}
// An output in its input's place has its strides.
int check_pair(const Rows& in, const Rows& out, int head_dim) {
    int rc = check_rows(in);
    if (rc == MOE_OK) rc = check_out(out, head_dim);
    if (rc == MOE_OK && in.p == out.p && (in.token != out.token || in.head != out.head)) rc = MOE_EINVAL;
    return rc;
}

void set_rows(moe::RotateParams& p, int i, const Rows& in, int heads) {
    p.src[i] = static_cast<const uint16_t*>(in.p);
    p.src_token[i] = in.token;
    p.src_head[i] = in.head;
    p.heads[i] = heads;
}
void set_out(moe::RotateParams& p, int i, const Rows& out) {
    p.dst[i] = static_cast<uint16_t*>(const_cast<void*>(out.p));
    p.dst_token[i] = out.token;
    p.dst_head[i] = out.head;
}
void set_angles(moe::RotateParams& p, const moe_rope_angles* a, const int32_t* positions) {
    p.positions = positions;
    p.turns = reinterpret_cast<const unsigned long long*>(a->turns);
    p.scale = a->scale;
    p.rotary_dim = a->rotary_dim;
    p.interleaved = a->interleaved;
}
template <class P>
void set_cache(P& p, const moe_kv_cache* c) {
    p.cache[0] = static_cast<uint8_t*>(c->k);
    p.cache[1] = static_cast<uint8_t*>(c->v);
    const int64_t s[2][3] = {{c->k_block_stride, c->k_token_stride, c->k_head_stride},
                             {c->v_block_stride, c->v_token_stride, c->v_head_stride}};
    for (int i = 0; i < 2; ++i) {
        p.cache_block[i] = 2 * s[i][0];
        p.cache_token[i] = 2 * s[i][1];
        p.cache_head[i] = 2 * s[i][2];
    }
    p.block_size = c->block_size;
    p.n_slots = (int64_t)c->n_blocks * c->block_size;
}
template <class P>
void set_cache(P& p, const moe_kv_cache8* c) {
    p.cache[0] = static_cast<uint8_t*>(c->k);
    p.cache[1] = static_cast<uint8_t*>(c->v);
    p.cache_scale[0] = c->k_scale;
    p.cache_scale[1] = c->v_scale;
    const int64_t s[2][3] = {{c->k_block_stride, c->k_token_stride, c->k_head_stride},
                             {c->v_block_stride, c->v_token_stride, c->v_head_stride}};
    for (int i = 0; i < 2; ++i) {
        p.cache_block[i] = s[i][0];
        p.cache_token[i] = s[i][1];
        p.cache_head[i] = s[i][2];
    }
    p.block_size = c->block_size;
    p.n_slots = (int64_t)c->n_blocks * c->block_size;
}

// Keys and values into a cache, rotated where there are angles, and queries
// rotated beside them.
template <class Cache>
int append(const Rows& q, const Rows& q_out, int q_heads, const Rows& k, const Rows& v, int T, int dtype,
           const int32_t* positions, const int32_t* slot_map, const moe_rope_angles* angles, bool rotate,
           const Cache* cache, int to, void* ws, size_t ws_bytes, void* stream) {
    if (T < 0 || (dtype != 0 && dtype != 1)) return MOE_ESHAPE;
    if (q_heads < 0 || q_heads > 1024) return MOE_ESHAPE;
    if (rotate) {
        const int rc = check_angles(angles, cache->head_dim);
        if (rc) return rc;
    }
    if (T == 0) return MOE_OK;
    if ((q.p != nullptr) != (q_heads > 0)) return MOE_ESHAPE;
    if (!slot_map || (rotate && !positions)) return MOE_EINVAL;
    int rc = check_rows(k);
    if (rc == MOE_OK) rc = check_rows(v);
    if (rc == MOE_OK && q_heads > 0) rc = check_pair(q, q_out, cache->head_dim);
    if (rc) return rc;
    if (!aligned4(slot_map) || !aligned4(positions)) return MOE_EALIGN;
    rc = check_ws(ws, ws_bytes, MOE_PAGED_WORKSPACE_BYTES);
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::RotateParams p = {};
    set_rows(p, 0, q, q_heads);
    set_rows(p, 1, k, cache->kv_heads);
    set_rows(p, 2, v, cache->kv_heads);
    set_out(p, 0, q_out);
    if (rotate) set_angles(p, angles, positions);
    set_cache(p, cache);
    p.slots = slot_map;
    p.ctrl = static_cast<unsigned*>(ws);
    p.T = T;
    p.head_dim = cache->head_dim;
    return launched(moe::launch_rotate(p, to, dtype, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

template <class Cache>
int read(const Cache* cache, const int32_t* slot_map, int T, int dtype, int from, const Rows& k, const Rows& v, void* ws,
         size_t ws_bytes, void* stream) {
    if (T < 0 || (dtype != 0 && dtype != 1)) return MOE_ESHAPE;
    if (T == 0) return MOE_OK;
    if (!slot_map) return MOE_EINVAL;
    int rc = check_out(k, cache->head_dim);
    if (rc == MOE_OK) rc = check_out(v, cache->head_dim);
    if (rc) return rc;
    if (!aligned4(slot_map)) return MOE_EALIGN;
    rc = check_ws(ws, ws_bytes, MOE_PAGED_WORKSPACE_BYTES);
    if (rc) return rc;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::ReadParams p = {};
    set_cache(p, cache);
    const Rows* out[2] = {&k, &v};
    for (int i = 0; i < 2; ++i) {
        p.dst[i] = static_cast<uint16_t*>(const_cast<void*>(out[i]->p));
        p.dst_token[i] = out[i]->token;
        p.dst_head[i] = out[i]->head;
    }
    p.slots = slot_map;
    p.ctrl = static_cast<unsigned*>(ws);
    p.T = T;
    p.heads = cache->kv_heads;
    p.lane_shift = cache->head_dim == 64 ? 2 : 3;
    return launched(moe::launch_read(p, from, dtype, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

// Tensor map of a cache of codes: (dimensions, token of the block, head, block),
// boxes of all dimensions of `box` tokens, swizzled by the dimensions' width. (The
// L2 fetches no more than a head's row: with 256 bytes at a time, the next head's
// row too, 4 tokens over 120,000 keys read half as much again from HBM.)
bool codes_map(CUtensorMap* m, const moe_kv_cache8* c, void* base, int64_t bs, int64_t ts, int64_t hs, int box) {
    const moe::EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->block_size, (cuuint64_t)c->kv_heads, (cuuint64_t)c->n_blocks};
    const cuuint64_t strides[3] = {(cuuint64_t)ts, (cuuint64_t)hs, (cuuint64_t)bs};
    const cuuint32_t boxes[4] = {(cuuint32_t)c->head_dim, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
               c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               c->head_dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

int moe_rope_turns(const double* radians, int n, uint64_t* turns) {
    if (n < 0) return MOE_ESHAPE;
    if (n > 0 && (!radians || !turns)) return MOE_EINVAL;
    for (int i = 0; i < n; ++i)
        if (!std::isfinite(radians[i])) return MOE_EINVAL;
    for (int i = 0; i < n; ++i) turns[i] = turns_of(radians[i]);
    return MOE_OK;
}

int moe_rope_table(int rotary_dim, double base, int scaling, double factor, int context, double low, double high,
                   uint64_t* turns, float* scale) {
    if (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > 512) return MOE_ESHAPE;
    if (!turns || !scale || scaling < MOE_ROPE_NONE || scaling > MOE_ROPE_BANDS) return MOE_EINVAL;
    if (!std::isfinite(base) || !(base > 1)) return MOE_EINVAL;
    const bool borders = scaling == MOE_ROPE_YARN || scaling == MOE_ROPE_BANDS;
    if (scaling != MOE_ROPE_NONE && (!std::isfinite(factor) || !(factor > 0))) return MOE_EINVAL;
    if (!std::isfinite(low) || !std::isfinite(high)) return MOE_EINVAL;
    if (low <= 0) low = 1;
    if (high <= 0) high = scaling == MOE_ROPE_YARN ? 32 : 4;
    if (borders && (context < 1 || !(low < high))) return MOE_EINVAL;
    const int pairs = rotary_dim / 2;
    // (factor^(pairs / (pairs - 1)) is the factor times a root of it)
    const Wide first_base = scaling == MOE_ROPE_NTK ? Wide(base) * factor * root_of(factor, pairs - 1) : Wide(base);
    if (!std::isfinite(first_base.hi) || !(first_base.hi > 0)) return MOE_EINVAL;
    // the pair's number at which a frequency makes n turns in the context
    auto pair_of = [&](double n) { return rotary_dim * std::log(context / (n * kTwoPi)) / (2 * std::log(base)); };
    double first = 0, last = 0;
    if (scaling == MOE_ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0);
        last = std::fmin(std::ceil(pair_of(low)), rotary_dim - 1);
    }
    const Wide ratio = Wide(1) / root_of(first_base, pairs);
    uint64_t own[256];
    Wide f = 1;
    for (int i = 0; i < pairs; ++i, f = f * ratio) {
        Wide kept = 1;  // share of the frequency that stays
        if (scaling == MOE_ROPE_LINEAR) kept = 0;
        if (scaling == MOE_ROPE_YARN) kept = Wide(1) + -(Wide(i - first) / std::fmax(last - first, 0.001));
        if (scaling == MOE_ROPE_BANDS) kept = (f * context / Wide(kTwoPi, kTwoPiLo) + -Wide(low)) / (Wide(high) + -Wide(low));
        if (kept.hi <= 0) kept = 0;
        if (kept.hi > 1 || (kept.hi == 1 && kept.lo >= 0)) kept = 1;
        const Wide scaled = kept.hi == 1 && kept.lo == 0 ? f : f / factor * (Wide(1) + -kept) + f * kept;
        if (!std::isfinite(scaled.hi + scaled.lo)) return MOE_EINVAL;
        own[i] = turns_of(scaled);
    }
    std::copy(own, own + pairs, turns);
    *scale = scaling == MOE_ROPE_YARN && factor > 1 ? (float)(0.1 * std::log(factor) + 1) : 1.f;
    return MOE_OK;
}

int moe_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t q_out_token_stride,
             int64_t q_out_head_stride, int q_heads, const void* k, int64_t k_token_stride, int64_t k_head_stride,
             void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride, int kv_heads, int T, int head_dim,
             int dtype, const int32_t* positions, const moe_rope_angles* angles, void* stream) {
    g_last_launches = 0;
    if (head_dim < 16 || head_dim % 16 != 0 || head_dim > 512 || (dtype != 0 && dtype != 1)) return MOE_ESHAPE;
    int rc = check_angles(angles, head_dim);
    if (rc) return rc;
    if (T < 0 || q_heads < 1 || q_heads > 1024 || kv_heads < 0 || kv_heads > 1024) return MOE_ESHAPE;
    if (T == 0) return MOE_OK;
    if ((k != nullptr) != (kv_heads > 0)) return MOE_ESHAPE;
    const Rows qs{q, q_token_stride, q_head_stride}, qo{q_out, q_out_token_stride, q_out_head_stride};
    const Rows ks{k, k_token_stride, k_head_stride}, ko{k_out, k_out_token_stride, k_out_head_stride};
    rc = check_pair(qs, qo, head_dim);
    if (rc == MOE_OK && k) rc = check_pair(ks, ko, head_dim);
    if (rc) return rc;
    if (!positions) return MOE_EINVAL;
    if (!aligned4(positions)) return MOE_EALIGN;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc) return rc;
    moe::RotateParams p = {};
    set_rows(p, 0, qs, q_heads);
    set_out(p, 0, qo);
    if (k) {
        set_rows(p, 1, ks, kv_heads);
        set_out(p, 1, ko);
    }
    set_angles(p, angles, positions);
    p.T = T;
    p.head_dim = head_dim;
    return launched(moe::launch_rotate(p, moe::kRotateRows, dtype, dev.sms, static_cast<cudaStream_t>(stream)), 1);
}

int moe_paged_rope_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                          int64_t q_out_token_stride, int64_t q_out_head_stride, int q_heads, const void* k_new,
                          int64_t k_token_stride, int64_t k_head_stride, const void* v_new, int64_t v_token_stride,
                          int64_t v_head_stride, int T, const int32_t* positions, const int32_t* slot_map,
                          const moe_rope_angles* angles, const moe_kv_cache* cache, void* ws, size_t ws_bytes,
                          void* stream) {
    g_last_launches = 0;
    const int rc = check_cache(cache);
    if (rc) return rc;
    return append({q, q_token_stride, q_head_stride}, {q_out, q_out_token_stride, q_out_head_stride}, q_heads,
                  {k_new, k_token_stride, k_head_stride}, {v_new, v_token_stride, v_head_stride}, T, cache->dtype, positions,
                  slot_map, angles, true, cache, moe::kRotateCache16, ws, ws_bytes, stream);
}

int moe_paged_rope_append8(const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                           int64_t q_out_token_stride, int64_t q_out_head_stride, int q_heads, const void* k_new,
                           int64_t k_token_stride, int64_t k_head_stride, const void* v_new, int64_t v_token_stride,
                           int64_t v_head_stride, int T, int dtype, const int32_t* positions, const int32_t* slot_map,
                           const moe_rope_angles* angles, const moe_kv_cache8* cache, void* ws, size_t ws_bytes,
                           void* stream) {
    g_last_launches = 0;
    const int rc = check_cache8(cache);
    if (rc) return rc;
    return append({q, q_token_stride, q_head_stride}, {q_out, q_out_token_stride, q_out_head_stride}, q_heads,
                  {k_new, k_token_stride, k_head_stride}, {v_new, v_token_stride, v_head_stride}, T, dtype, positions,
                  slot_map, angles, true, cache, moe::kRotateCache8, ws, ws_bytes, stream);
}

int moe_paged_append8(const void* k_new, int64_t k_token_stride, int64_t k_head_stride, const void* v_new,
                      int64_t v_token_stride, int64_t v_head_stride, int T, int dtype, const int32_t* slot_map,
                      const moe_kv_cache8* cache, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    const int rc = check_cache8(cache);
    if (rc) return rc;
    return append({nullptr, 0, 0}, {nullptr, 0, 0}, 0, {k_new, k_token_stride, k_head_stride},
                  {v_new, v_token_stride, v_head_stride}, T, dtype, nullptr, slot_map, nullptr, false, cache,
                  moe::kRotateCache8, ws, ws_bytes, stream);
}

int moe_paged_read(const moe_kv_cache* cache, const int32_t* slot_map, int T, void* k_out, int64_t k_token_stride,
                   int64_t k_head_stride, void* v_out, int64_t v_token_stride, int64_t v_head_stride, void* ws,
                   size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    const int rc = check_cache(cache);
    if (rc) return rc;
    return read(cache, slot_map, T, cache->dtype, 0, {k_out, k_token_stride, k_head_stride},
                {v_out, v_token_stride, v_head_stride}, ws, ws_bytes, stream);
}

int moe_paged_read8(const moe_kv_cache8* cache, const int32_t* slot_map, int T, int dtype, void* k_out,
                    int64_t k_token_stride, int64_t k_head_stride, void* v_out, int64_t v_token_stride,
                    int64_t v_head_stride, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    const int rc = check_cache8(cache);
    if (rc) return rc;
    return read(cache, slot_map, T, dtype, 1, {k_out, k_token_stride, k_head_stride},
                {v_out, v_token_stride, v_head_stride}, ws, ws_bytes, stream);
}

size_t moe_paged_attention8_workspace_bytes(int q_heads, const moe_kv_cache8* cache) {
    if (check_cache8(cache) != MOE_OK) return 0;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > 32) return 0;
    return MOE_PAGED_WORKSPACE_BYTES + 3 * MOE_MAX_GRID * sizeof(unsigned) +
           (size_t)MOE_MAX_GRID * 2 * moe::attn_part_floats(moe::kAttnRows, cache->head_dim) * sizeof(float);
}

int moe_paged_attention8(const void* q, int64_t q_token_stride, int64_t q_head_stride, int T, int q_heads, int dtype,
                         const moe_kv_cache8* cache, const int32_t* block_tables, int max_blocks, const int32_t* q_start,
                         const int32_t* seq_lens, const uint64_t* masks, int B, float scale, int window, void* out,
                         float* lse, void* ws, size_t ws_bytes, void* stream) {
    g_last_launches = 0;
    int rc = check_cache8(cache);
    if (rc) return rc;
    if (dtype != 0 && dtype != 1) return MOE_ESHAPE;
    if (q_heads < 1 || q_heads % cache->kv_heads != 0 || q_heads / cache->kv_heads > 32) return MOE_ESHAPE;
    const int group = q_heads / cache->kv_heads;
    if (T < 0 || (int64_t)T * group >= (1 << 28)) return MOE_ESHAPE;
    if (B < 1 || B > MOE_PAGED_MAX_REQUESTS || max_blocks < 1 || window < 0 || (masks && window > 0)) return MOE_ESHAPE;
    if (!(scale == scale) || std::isinf(scale)) return MOE_EINVAL;
    if (!block_tables || !q_start || !seq_lens) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!out) return MOE_EINVAL;
    rc = check_rows({q, q_token_stride, q_head_stride});
    if (rc) return rc;
    if (!aligned16(out) || !aligned4(lse) || !aligned4(block_tables) || !aligned4(q_start) || !aligned4(seq_lens) ||
        !aligned8(masks))
        return MOE_EALIGN;
    rc = check_ws(ws, ws_bytes, moe_paged_attention8_workspace_bytes(q_heads, cache));
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
    // (behind all the counters of the attention over 16 bits, which a workspace that
    // serves both keeps zero between calls)
    p.part = reinterpret_cast<float*>(p.arrived + 3 * MOE_MAX_GRID);
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
    p.scales[0] = cache->k_scale;
    p.scales[1] = cache->v_scale;
    CUtensorMap k_map, v_map;
    if (!codes_map(&k_map, cache, cache->k, cache->k_block_stride, cache->k_token_stride, cache->k_head_stride, p.box) ||
        !codes_map(&v_map, cache, cache->v, cache->v_block_stride, cache->v_token_stride, cache->v_head_stride, p.box))
        return MOE_ECUDA;
    return launched(moe::launch_attn_codes(p, &k_map, &v_map, cache->head_dim, dtype, static_cast<cudaStream_t>(stream)), 1);
}

}  // extern "C"
