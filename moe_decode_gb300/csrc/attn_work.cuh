// Attention over the paged cache: the requests' lengths, the division of the
// work over the CTAs, and which keys and boxes of the cache a row or a tile
// needs. Integer arithmetic alone, which a host compiler takes too
// (tests/attn_work_host.cpp).
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
#include "layer_params.h"
#include "paged.h"

namespace moe {

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

// The first key that a row at position pos sees. (Without a step past 32 bits,
// however wide the window and however far below zero the position: an overflow
// is undefined, and the counts of units of the CTAs' roles then need not agree.)
// (A selection by pos >= window instead of the two maxima costs the chunk kernel
// 1%, by the registers of its other loops.)
__device__ __forceinline__ int first_seen(const AttnParams& p, int pos) {
    return p.window > 0 ? max(max(pos, 0) - p.window + 1, 0) : 0;
}

// Keys [lo, hi) that the rows [row0, row0 + rows) of a request see between
// them, inside the block table; `over` where a row sees past it.
__device__ __forceinline__ void attn_keys(const AttnParams& p, const Request& q, int row0, int rows, int& lo, int& hi,
                                          bool& over) {
    const int first = q.pos0 + token_of(p, row0), last = q.pos0 + token_of(p, row0 + rows - 1);
    const int64_t cap = (int64_t)p.max_blocks * p.block_size;
    over = last + 1 > cap;
    hi = (int)min((int64_t)last + 1, cap);
    lo = first_seen(p, first);
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
        return attn_tiles(first_seen(p, pos0 + first), hi);
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

// The CTA's range of the call's at.total units.
__device__ __forceinline__ void attn_range(const AttnParams& p, int cta, Place& at) {
    at.ctas = (int)min((int64_t)p.G, at.total);
    at.begin = cta < at.ctas ? scaled(at.total, cta, at.ctas) : at.total;
    at.end = cta < at.ctas ? scaled(at.total, cta + 1, at.ctas) : at.total;
}

// The item of unit `rest` (there is one) of the requests [r0, r1).
template <class Class>
__device__ __forceinline__ Start attn_seek(const AttnParams& p, int r0, int r1, int64_t rest) {
    for (int r = r0; r < r1; ++r) {
        const Request q = attn_request(p, r);
        const int64_t per_head = Class::mine(p, q) ? attn_request_units<Class>(p, q) : 0;
        if (rest >= per_head * p.kv_heads) {
            rest -= per_head * p.kv_heads;
            continue;
        }
        const int head = rest < (1 << 30) && per_head < (1 << 30) ? (int)((uint32_t)rest / (uint32_t)per_head)
                                                                  : (int)(rest / per_head);
        rest -= head * per_head;
        RowTiles<Class::kRows> t(p, q);
        for (int u = Class::kItem + t.tiles(); rest >= u; u = Class::kItem + t.tiles()) {
            rest -= u;
            t.next();
        }
        return Start{r, head, t.row0, (int)rest, q};
    }
    return Start{};
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

// The keys that row `row` of the item at hand sees, [from, last] (from > last:
// none). Rows past its end see none.
struct RowKeys {
    int last, from;
};
template <class W>
__device__ __forceinline__ RowKeys attn_row_keys(const W& walk, int row) {
    const int pos = walk.q.pos0 + token_of(walk.p, walk.row0 + min(row, walk.rows - 1));
    return RowKeys{row < walk.rows ? min(pos, walk.hi - 1) : -1, first_seen(walk.p, pos)};
}
// Keys that all rows [from, to) of it see: [all_from, all_to).
struct AllKeys {
    int to, from;
    // whether some row does not see one of the keys [key, key + n)
    __device__ __forceinline__ bool lacks(int key, int n) const { return key > to - n || key < from; }
};
template <class W>
__device__ __forceinline__ AllKeys attn_all_keys(const W& walk, int from, int to) {
    return AllKeys{min(walk.q.pos0 + token_of(walk.p, walk.row0 + from) + 1, walk.hi),
                   first_seen(walk.p, walk.q.pos0 + token_of(walk.p, walk.row0 + to - 1))};
}
// Of the keys [key, key + n) (key >= 0): whether the item needs any, and
// whether there are some that it does not.
template <class W>
__device__ __forceinline__ bool attn_needs(const W& walk, int key, int n) { return key < walk.hi && key > walk.lo - n; }
template <class W>
__device__ __forceinline__ bool attn_ragged(const W& walk, int key, int n) { return key < walk.lo || key > walk.hi - n; }

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
        // (a tile may end at key 2^31: no lane goes past it, and no sum reaches it)
        const int key = (walk.tile0 + t) * kAttnTile + min(lane * p.box, kAttnTile - p.box);
        b.wanted = any && lane < kAttnTile / p.box && key < walk.hi && key > walk.lo - p.box;
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

}  // namespace moe
