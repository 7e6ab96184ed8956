// What the kernels of attention over the paged cache share: the requests'
// lengths, the division of the work over the CTAs, bounded waits, tensor-map
// copies of pages.
//
// An item is up to ROWS query rows of one request and one kv head: row R of a
// request is token R / group, query head R % group of the kv head's group, so
// that the heads that share keys share the read. A unit is one tile of
// kAttnTile keys of one item. All units of the call in the order request, kv
// head, row tile, key tile are divided evenly: of G CTAs (or as many as there
// are units) CTA c takes the units [cU/G, (c+1)U/G), whatever the lengths. An
// item's first units stand for what it costs beside its tiles (queries, joining
// warps, output): a batch of short requests would otherwise be unevenly spread. An item whose units all lie in one CTA is
// finished there; of one that spans CTAs each leaves its part (unnormalised
// sums, largest score, sum of weights) in the workspace, and the CTA that comes
// last joins the parts, in the order of the keys whoever it is.
#pragma once
#include <cuda.h>

#include "layer_params.h"
#include "paged.h"
#include "ptx.cuh"

namespace moe {

constexpr float kLn2 = 0.693147180559945f;

// The token of a query row within its request.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
    return (int)(((unsigned long long)(unsigned)row * p.group_magic) >> 36);
}

// a * b / c, in 32 bits where that suffices (a 64-bit division takes some 400
// cycles, and a call with few units waits for each).
__device__ __forceinline__ int64_t scaled(int64_t a, int b, int64_t c) {
    if (a < (1 << 22) && c < (1 << 22)) return (uint32_t)a * (uint32_t)b / (uint32_t)c;  // b <= 256 CTAs
    return a * b / c;
}

struct Request {
    int q0, n;     // first token row, tokens
    int pos0;      // position of the first token (negative: rows that see nothing)
    bool bad;
};

__device__ __forceinline__ Request attn_request(const AttnParams& p, int r) {
    Request q;
    // (past the L1: the chunk kernel begins without a wait of its own)
    const int a = __ldcg(p.q_start + r), b = __ldcg(p.q_start + r + 1);
    const int seq = __ldcg(p.seq + r);
    q.bad = a < 0 || b < a || b > p.T || seq < 0;
    q.q0 = a;
    q.n = q.bad ? 0 : b - a;
    q.pos0 = q.bad ? 0 : seq - q.n;
    return q;
}

// Keys [lo, hi) that the rows [row0, row0 + rows) of a request see between
// them, inside the block table; `over` where a row sees past it.
__device__ __forceinline__ void attn_keys(const AttnParams& p, const Request& q, int row0, int rows, int& lo, int& hi,
                                          bool& over) {
    const int first = q.pos0 + token_of(p, row0), last = q.pos0 + token_of(p, row0 + rows - 1);
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    over = last + 1 > cap;
    hi = (int)min((int64_t)last + 1, cap);
    lo = p.window > 0 ? max(first - p.window + 1, 0) : 0;
    if (hi <= lo) lo = hi = 0;
}

// Units of one row tile. A row tile without keys is one unit: its rows are
// written all the same.
__device__ __forceinline__ int attn_tiles(int lo, int hi) {
    return hi > lo ? (hi - 1) / kAttnTile - lo / kAttnTile + 1 : 1;
}

// The row tiles of a request in order: units of each, with the token of a
// tile's first and last row kept by addition (a chunk of 8,192 tokens has some
// hundred row tiles, and one thread counts them).
template <int ROWS>
struct RowTiles {
    const AttnParams& p;
    int pos0, rows, row0 = 0;
    int first, first_rem;  // token of the tile's first row, row within the token
    int step, step_rem;
    int64_t cap;
    __device__ __forceinline__ RowTiles(const AttnParams& params, const Request& q)
        : p(params), pos0(q.pos0), rows(q.n * params.group), first(0), first_rem(0), step(token_of(params, ROWS)),
          step_rem(ROWS - token_of(params, ROWS) * params.group), cap((int64_t)params.max_blocks * params.block_size) {}
    __device__ __forceinline__ bool more() const { return row0 < rows; }
    __device__ __forceinline__ int tiles() const {
        int last = first + step + (first_rem + step_rem >= p.group ? 1 : 0);  // token of the next tile's first row
        if (first_rem + step_rem == 0 || first_rem + step_rem == p.group) --last;  // which may begin there
        if (row0 + ROWS >= rows) last = token_of(p, rows - 1);
        const int hi = (int)min((int64_t)pos0 + last + 1, cap);
        const int lo = p.window > 0 ? max(pos0 + first - p.window + 1, 0) : 0;
        return attn_tiles(lo, hi);
    }
    __device__ __forceinline__ void next() {
        row0 += ROWS;
        first += step;
        first_rem += step_rem;
        if (first_rem >= p.group) {
            first_rem -= p.group;
            ++first;
        }
    }
};

// Units of a request for one kv head.
template <class Class>
__device__ __forceinline__ int64_t attn_request_units(const AttnParams& p, const Request& q) {
    int64_t u = 0;
    for (RowTiles<Class::kRows> t(p, q); t.more(); t.next()) u += Class::kItem + t.tiles();
    return u;
}

// Which kernel takes a request, the rows of its items, and the units that an
// item costs beside its tiles.
struct Few {
    static constexpr int kRows = kAttnRows, kItem = 2;
    static __device__ __forceinline__ bool mine(const AttnParams& p, const Request& q) {
        return q.n > 0 && q.n * p.group <= kAttnFewRows;
    }
};
struct Many {
    static constexpr int kRows = kAttnChunkRows, kItem = 2;
    static __device__ __forceinline__ bool mine(const AttnParams& p, const Request& q) {
        return q.n * p.group > kAttnFewRows;
    }
};

// A place in the order of units, and the CTA's range.
struct Start {
    int request, head, row0;
    int skip;  // units of that item before the range
    Request q;
};
struct Place {
    int64_t total;      // units of the call
    int ctas;           // CTAs with units
    int64_t begin, end; // this CTA's
    Start start;        // the item of unit `begin`
};

// Finds the CTA's range and the item that it begins in, all threads together:
// one of them walks to the item, for all. `scan` is shared memory of THREADS /
// 32 values.
template <class Class, int THREADS>
__device__ __forceinline__ Place attn_place(const AttnParams& p, int cta, int64_t* scan, Start* found) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);
    int64_t own = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Request q = attn_request(p, r);
        bad |= q.bad;
        if (Class::mine(p, q)) own += attn_request_units<Class>(p, q) * p.kv_heads;
    }
    if (bad) atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
    int64_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    Place at;
    at.total = 0;
    int64_t before = sum - own;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scan[w];
        at.total += scan[w];
    }
    at.ctas = (int)min((int64_t)p.G, at.total);
    at.begin = cta < at.ctas ? scaled(at.total, cta, at.ctas) : at.total;
    at.end = cta < at.ctas ? scaled(at.total, cta + 1, at.ctas) : at.total;
    if (own > 0 && before <= at.begin && at.begin < before + own) {
        for (int r = r0; r < r1; ++r) {
            const Request q = attn_request(p, r);
            const int64_t per_head = Class::mine(p, q) ? attn_request_units<Class>(p, q) : 0;
            if (at.begin < before + per_head * p.kv_heads) {
                int64_t rest = at.begin - before;
                const int head = rest < (1 << 30) && per_head < (1 << 30) ? (int)((uint32_t)rest / (uint32_t)per_head)
                                                                          : (int)(rest / per_head);
                rest -= head * per_head;
                RowTiles<Class::kRows> t(p, q);
                for (int u = Class::kItem + t.tiles(); rest >= u; u = Class::kItem + t.tiles()) {
                    rest -= u;
                    t.next();
                }
                *found = Start{r, head, t.row0, (int)rest, q};
                break;
            }
            before += per_head * p.kv_heads;
        }
    }
    __syncthreads();
    at.start = *found;  // (anything, for a CTA without units)
    return at;
}

// The items of a CTA's range, one after another; every role of the CTA walks
// them alike.
template <class Class>
struct Walk {
    static constexpr int ROWS = Class::kRows;
    const AttnParams& p;
    int64_t unit, end;  // next unit of the range
    int r, head, row0;
    int skip;           // units of the item at hand before the range
    Request q;
    // the item at hand
    int rows, lo, hi, tile0, tiles;
    int t0, t1;         // its tiles [t0, t1) in this range
    bool over;

    __device__ __forceinline__ Walk(const AttnParams& params, const Place& at)
        : p(params), unit(at.begin), end(at.end), r(at.start.request), head(at.start.head), row0(at.start.row0),
          skip(at.start.skip), q(at.start.q) {}
    __device__ __forceinline__ void item() {
        rows = min(ROWS, q.n * p.group - row0);
        attn_keys(p, q, row0, rows, lo, hi, over);
        tile0 = lo / kAttnTile;
        tiles = attn_tiles(lo, hi);
    }
    // The next item with tiles in the range into the fields; false at the end.
    __device__ __forceinline__ bool next() {
        if (unit >= end) return false;
        item();
        t0 = max(skip - Class::kItem, 0);
        t1 = (int)min((int64_t)tiles, skip - Class::kItem + (end - unit));
        return t1 > t0;  // (only the last item may have none)
    }
    __device__ __forceinline__ void done() {
        unit += Class::kItem + tiles - skip;
        skip = 0;
        if (unit >= end) return;
        row0 += ROWS;
        if (row0 < q.n * p.group) return;
        row0 = 0;
        if (++head < p.kv_heads) return;
        head = 0;
        do {
            q = attn_request(p, ++r);
        } while (!Class::mine(p, q));
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // An item that began in an earlier CTA leaves part 0, one that goes on in
    // the next CTA part 1.
    __device__ __forceinline__ int part() const { return t0 > 0 ? 0 : 1; }
};

// The CTA in which an item's first tile lies, and how many CTAs hold its tiles
// (the CTA of unit u is the largest k with kU/G <= u).
struct Span {
    int cta, parts;
};
__device__ __forceinline__ int cta_of(int64_t unit, const Place& at) {
    if (at.total < (1 << 22)) return (int)(((uint32_t)(unit + 1) * (uint32_t)at.ctas - 1) / (uint32_t)at.total);
    return (int)(((unit + 1) * at.ctas - 1) / at.total);
}
template <class Class>
__device__ __forceinline__ Span attn_span(const Walk<Class>& walk, const Place& at) {
    const int64_t u = walk.unit - walk.skip + Class::kItem;
    Span s;
    s.cta = cta_of(u, at);
    s.parts = cta_of(u + walk.tiles - 1, at) - s.cta + 1;
    return s;
}

// One thread of a CTA whose part is in place (its threads' stores are behind a
// barrier): whether all the others are. The last one to come leaves the count
// at zero for the next call.
__device__ __forceinline__ bool attn_last(unsigned* arrived, int parts) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(arrived) : "memory");
    if (old != (unsigned)parts - 1) return false;
    asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(arrived) : "memory");
    return true;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
__device__ __forceinline__ float exp2_approx(float x);

// (A sum of weights is 0, NaN or above 0: NaN has to reach the output and lse.)
// Joins the parts of an item, in the order of the keys (the part 1 of the CTA
// that it begins in, then the part 0 of the CTAs after it): THREADS threads,
// the rows [from, to). A thread takes U pieces of 8 dimensions at a time, all
// their loads of a part in flight together.
template <int D, int DT, int ROWS, int THREADS, int U>
__device__ __forceinline__ void attn_join(const AttnParams& p, const float* parts, const Span& span, int from, int to,
                                          int row0, int head, int token0, int tid) {
    constexpr int kFloats = attn_part_floats(ROWS, D), kPer = D / 8;
    const float* first = parts + ((int64_t)span.cta * 2 + 1) * kFloats;
    const float* rest = parts + (int64_t)span.cta * 2 * kFloats;  // part 0 of the k-th CTA at k * 2 * kFloats
    auto part_of = [&](int k) { return k == 0 ? first : rest + (int64_t)k * 2 * kFloats; };
    auto stat_of = [&](int k, int row) { return __ldcg(reinterpret_cast<const float2*>(part_of(k) + ROWS * D) + row); };
    const int end = to * kPer;
    for (int i0 = tid + from * kPer; i0 < end; i0 += U * THREADS) {
        // (past the end the last piece again, not stored)
        float mx[U], sum[U], v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mx[u] = -INFINITY;
            sum[u] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
        }
#pragma unroll 2
        for (int k = 0; k < span.parts; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) mx[u] = fmaxf(mx[u], stat_of(k, min(i0 + u * THREADS, end - 1) / kPer).x);
        for (int k = 0; k < span.parts; ++k) {
            float2 ml[U];
            float4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = min(i0 + u * THREADS, end - 1);
                const float4* f = reinterpret_cast<const float4*>(part_of(k) + (int64_t)i * 8);
                ml[u] = stat_of(k, i / kPer);
                x[u] = __ldcg(f);
                y[u] = __ldcg(f + 1);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = exp2_approx(ml[u].x - (mx[u] == -INFINITY ? 0.f : mx[u]));
                sum[u] += w * ml[u].y;
                v[u][0] += w * x[u].x; v[u][1] += w * x[u].y; v[u][2] += w * x[u].z; v[u][3] += w * x[u].w;
                v[u][4] += w * y[u].x; v[u][5] += w * y[u].y; v[u][6] += w * y[u].z; v[u][7] += w * y[u].w;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * THREADS;
            if (i >= end) break;
            const int row = i / kPer, d = (i % kPer) * 8;
            const float inv = sum[u] != 0.f ? 1.f / sum[u] : 0.f;
            const int R = row0 + row, t = token_of(p, R), h = head * p.group + (R - t * p.group);
            const int64_t at_row = (int64_t)(token0 + t) * p.heads + h;
            uint4 o;
            o.x = pack2<DT>(v[u][0] * inv, v[u][1] * inv);
            o.y = pack2<DT>(v[u][2] * inv, v[u][3] * inv);
            o.z = pack2<DT>(v[u][4] * inv, v[u][5] * inv);
            o.w = pack2<DT>(v[u][6] * inv, v[u][7] * inv);
            *reinterpret_cast<uint4*>(p.out + at_row * D + d) = o;
            if (d == 0 && p.lse) p.lse[at_row] = sum[u] != 0.f ? (mx[u] + log2f(sum[u])) * kLn2 : -INFINITY;
        }
    }
}

// A part of the chunk kernel: for each slot of 128 rows four dimensions of all
// rows after another, so that a warp's 32 rows are stored and read together;
// then the rows' largest scores and sums. The join, a thread a row: bound by
// what one SM reads from the L2 (two slots of 128 dimensions in five parts,
// 640 KB, take 14,000 cycles; 33,000 with rows of the part side by side).
template <int D, int DT>
__device__ __noinline__ void attn_join_slot(const AttnParams& p, const float* parts, const Span& span, int slot, int row,
                                               int64_t at_row, bool real) {
    constexpr int kFloats = attn_part_floats(kAttnChunkRows, D), kSlot = 128;
    const float* first = parts + ((int64_t)span.cta * 2 + 1) * kFloats;
    const float* rest = parts + (int64_t)span.cta * 2 * kFloats;  // part 0 of the k-th CTA at k * 2 * kFloats
    auto part_of = [&](int k) { return k == 0 ? first : rest + (int64_t)k * 2 * kFloats; };
    auto stat_of = [&](int k) {
        return __ldcg(reinterpret_cast<const float2*>(part_of(k) + kAttnChunkRows * D) + slot * kSlot + row);
    };
    float mx = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < span.parts; ++k) mx = fmaxf(mx, stat_of(k).x);
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int k = 0; k < span.parts; ++k) {
        const float2 ml = stat_of(k);
        sum += exp2_approx(ml.x - ref) * ml.y;
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    constexpr int kStep = 16;  // 16-byte loads in flight
#pragma unroll
    for (int c0 = 0; c0 < D / 4; c0 += kStep) {
        float4 v[kStep];
#pragma unroll
        for (int c = 0; c < kStep; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < span.parts; ++k) {
            const float4* f = reinterpret_cast<const float4*>(part_of(k)) + (slot * (D / 4) + c0) * kSlot + row;
            float4 x[kStep];
#pragma unroll
            for (int c = 0; c < kStep; ++c) x[c] = __ldcg(f + c * kSlot);
            const float w = exp2_approx(stat_of(k).x - ref) * inv;
#pragma unroll
            for (int c = 0; c < kStep; ++c) {
                v[c].x += w * x[c].x;
                v[c].y += w * x[c].y;
                v[c].z += w * x[c].z;
                v[c].w += w * x[c].w;
            }
        }
        if (!real) continue;
#pragma unroll
        for (int c = 0; c < kStep; c += 2) {
            uint4 o;
            o.x = pack2<DT>(v[c].x, v[c].y);
            o.y = pack2<DT>(v[c].z, v[c].w);
            o.z = pack2<DT>(v[c + 1].x, v[c + 1].y);
            o.w = pack2<DT>(v[c + 1].z, v[c + 1].w);
            *reinterpret_cast<uint4*>(p.out + at_row * D + (c0 + c) * 4) = o;
        }
    }
    if (real && p.lse) p.lse[at_row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Waits for the phase with parity `parity`, at most timeout_ns; false, with
// the status and `flag` set, when it ran out or another wait of the CTA did.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, const AttnParams& p, volatile int* flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*flag) return false;
        if (global_timer_ns() - t0 > p.timeout_ns) {
            atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -101 /* MOE_ETIMEOUT */);
            *flag = 1;
            return false;
        }
    }
    return true;
}

// One box of a cache's tensor map (64 dimensions, token of the block, which 64,
// head, block) into shared memory: `box` keys, 128 bytes a key in the 128-byte
// swizzle, one panel of 64 dimensions after another. The innermost coordinate
// is always 0.
__device__ __forceinline__ void attn_copy(uint32_t dst, const CUtensorMap* map, int panel, int token, int head,
                                          int block, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(0), "r"(token), "r"(panel), "r"(head), "r"(block), "r"(bar)
        : "memory");
}

// The producers' order of tiles: the box that this lane brings of the tile at
// hand. The block number is asked for one tile ahead of its use.
template <class Class>
struct TileFeed {
    Walk<Class> walk;
    int t, lane;
    bool any;  // whether the range has a tile
    __device__ __forceinline__ TileFeed(const AttnParams& p, const Place& at, int l) : walk(p, at), t(0), lane(l) {
        any = walk.next();
        if (any) start();
    }
    __device__ __forceinline__ void start() {
        t = walk.t0;
        if (walk.over && lane == 0)
            atomicCAS(reinterpret_cast<int*>(walk.p.ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
    }
    struct Box {
        int block, token, head;
        bool wanted;  // a row sees some of it
        // with the item's first tile: its rows, the first of them, and the
        // request's first token row (else rows is 0)
        int rows, row0, token0;
    };
    __device__ __forceinline__ Box box() const {
        const AttnParams& p = walk.p;
        Box b;
        const int key = (walk.tile0 + t) * kAttnTile + lane * p.box;
        b.wanted = any && lane < kAttnTile / p.box && key < walk.hi && key + p.box > walk.lo;
        b.head = walk.head;
        b.rows = any && t == walk.t0 ? walk.rows : 0;
        b.row0 = walk.row0;
        b.token0 = walk.q.q0;
        b.block = b.token = 0;
        if (b.wanted) {
            const int page = key / p.block_size;
            b.token = key - page * p.block_size;
            b.block = __ldcg(p.tables + (int64_t)walk.r * p.max_blocks + page);
        }
        return b;
    }
    __device__ __forceinline__ bool advance() {  // false after the last tile
        if (++t < walk.t1) return true;
        walk.done();
        if (!walk.next()) return false;
        start();
        return true;
    }
};
// Whether the box is copied: wanted and in a block that there is.
__device__ __forceinline__ bool attn_take(const AttnParams& p, bool wanted, int block) {
    if (wanted && (unsigned)block >= (unsigned)p.n_blocks) {
        atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
        return false;
    }
    return wanted;
}

// The softmax weights are 2^(score - m). The reference m of a row is set kBias
// below its largest score and stays until a score is more than kLimit above it,
// so most tiles need no pass over the sums. bf16 has fp32's exponents. fp16 ends
// at 2^-24: next to a largest weight of 1 many keys of 2^-25 each would be lost
// (60,000 of them are 0.2% of the output), so its weights reach up to 2^15 and
// the least that it holds is 2^-35 of the largest.
template <int DT>
struct WeightRange {
    static constexpr float kBias = DT == 0 ? 0.f : 11.f, kLimit = DT == 0 ? 8.f : 15.f;
};

// Two fp32 into one register of the type, `lo` in the low half (one rounding).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    if (DT == 0) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace moe
