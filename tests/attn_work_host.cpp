// The division of the paged attention's work, run by a host compiler over the
// requests of the command line: every tile of every item has to lie in exactly
// one CTA, be made of the keys that its rows see, and no load may leave its
// array. Built with a trap on signed overflow (tests/test_attn_work.py).
//
//   attn_work_host page window max_blocks kv_heads group ctas seq,new ...
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

static void fail(const char* what) {
    std::printf("%s\n", what);
    std::exit(1);
}

// The arrays that the code under test may read.
struct Span32 {
    const int32_t* at;
    size_t n;
};
static std::vector<Span32> readable;
static int32_t __ldcg(const int32_t* p) {
    for (const Span32& s : readable)
        if (p >= s.at && p < s.at + s.n) return *p;
    fail("a load outside its array");
    return 0;
}
static int atomicCAS(int* p, int, int v) { return *p = v; }
using std::max;
using std::min;

#include "attn_work.cuh"

using namespace moe;

template <class Class>
static void check(AttnParams p, const std::vector<std::pair<int64_t, int64_t>>& lens) {
    constexpr int ROWS = Class::kRows;
    Place at = {};
    for (int r = 0; r < p.B; ++r) {
        const Request q = attn_request(p, r);
        if (Class::mine(p, q)) at.total += attn_request_units<Class>(p, q) * p.kv_heads;
    }
    if (at.total < 0) fail("negative work");
    // tiles that have been seen of each item, and its row tiles
    std::map<std::tuple<int, int, int>, int> seen;
    for (int cta = 0; cta < p.G; ++cta) {
        attn_range(p, cta, at);
        if (at.begin >= at.end) continue;
        at.start = attn_seek<Class>(p, 0, p.B, at.begin);
        for (Walk<Class> w(p, at); w.next(); w.done()) {
            if (w.r < 0 || w.r >= p.B) fail("a request that is not there");
            const int64_t seq = lens[w.r].first, n = lens[w.r].second, first = seq - n + w.row0 / p.group,
                          last = seq - n + (w.row0 + std::min<int64_t>(ROWS, n * p.group - w.row0) - 1) / p.group;
            int64_t hi = std::min(last + 1, (int64_t)p.max_blocks * p.block_size),
                    lo = p.window > 0 ? std::max<int64_t>(first - p.window + 1, 0) : 0;
            if (hi <= lo) lo = hi = 0;
            if (w.lo != lo || w.hi != hi) fail("other keys than the rows see");
            if (w.tiles != (hi > lo ? (hi - 1) / kAttnTile - lo / kAttnTile + 1 : 1)) fail("other tiles than the keys'");
            if (w.t0 < 0 || w.t1 > w.tiles) fail("tiles that are not there");
            int& done = seen[{w.r, w.head, w.row0}];
            if (done != w.t0) fail("a tile left out or taken twice");
            done = w.t1;
            // what the rows see of each tile, in quarters too
            auto seen_from = [&](int64_t pos) { return p.window > 0 ? std::max<int64_t>(pos - p.window + 1, 0) : 0; };
            for (int row = 0; row < ROWS; ++row) {
                const int64_t pos = seq - n + (w.row0 + row) / p.group;
                const RowKeys k = attn_row_keys(w, row);
                if (row >= w.rows ? k.last >= 0 : k.last != std::min(pos, hi - 1) || k.from != seen_from(pos))
                    fail("other keys than the row sees");
            }
            for (int from = 0; from < w.rows; from += 128) {
                const int to = min(from + 128, w.rows);
                const AllKeys all = attn_all_keys(w, from, to);
                for (int t = w.t0; t < w.t1; ++t)
                    for (int n_keys : {32, kAttnTile})
                        for (int64_t key = (int64_t)(w.tile0 + t) * kAttnTile, end = key + kAttnTile; key < end; key += n_keys) {
                            const int64_t first_pos = seq - n + (w.row0 + from) / p.group, last_pos = seq - n + (w.row0 + to - 1) / p.group;
                            if (all.lacks((int)key, n_keys) !=
                                (key + n_keys > std::min(first_pos + 1, hi) || key < seen_from(last_pos)))
                                fail("a row's missing keys not noticed");
                            if (attn_needs(w, (int)key, n_keys) != (key < hi && key + n_keys > lo) ||
                                attn_ragged(w, (int)key, n_keys) != (key < lo || key + n_keys > hi))
                                fail("an item's keys not noticed");
                        }
            }
            const Span s = attn_span(w, at);
            if (cta < s.cta || cta >= s.cta + s.parts) fail("a part outside its item's CTAs");
            if (w.whole() != (s.parts == 1)) fail("a count of parts that is not the item's");
        }
        // the boxes of all lanes
        std::vector<TileFeed<Class>> feed;
        for (int lane = 0; lane < 32; ++lane) feed.emplace_back(p, at, lane);
        for (bool more = feed[0].any; more;) {
            const int64_t key0 = (int64_t)(feed[0].walk.tile0 + feed[0].t) * kAttnTile;
            for (int lane = 0; lane < 32; ++lane) {
                const auto box = feed[lane].box();
                const int64_t key = key0 + (int64_t)lane * p.box;
                const bool want = lane < kAttnTile / p.box && key < feed[0].walk.hi && key + p.box > feed[0].walk.lo;
                if (box.wanted != want) fail("a box that is not needed, or is missing");
                if (want && box.token != key % p.block_size) fail("another token of the block");
            }
            for (auto& f : feed) more = f.advance();
        }
    }
    size_t items = 0;
    for (int r = 0; r < p.B; ++r) {
        const Request q = attn_request(p, r);
        if (!Class::mine(p, q)) continue;
        for (int row0 = 0; row0 < q.n * p.group; row0 += ROWS, ++items) {
            int lo, hi;
            bool over;
            attn_keys(p, q, row0, min(ROWS, q.n * p.group - row0), lo, hi, over);
            for (int head = 0; head < p.kv_heads; ++head)
                if (seen[{r, head, row0}] != attn_tiles(lo, hi)) fail("an item that is not finished");
        }
    }
    if (seen.size() != items * p.kv_heads) fail("items that are not there");
}

int main(int argc, char** argv) {
    AttnParams p = {};
    p.block_size = std::atoi(argv[1]);
    p.window = std::atoi(argv[2]);
    p.max_blocks = std::atoi(argv[3]);
    p.kv_heads = std::atoi(argv[4]);
    p.group = std::atoi(argv[5]);
    p.G = std::atoi(argv[6]);
    p.heads = p.kv_heads * p.group;
    p.group_magic = ((1ull << 36) + p.group - 1) / p.group;
    p.box_shift = std::min(__builtin_ctz((unsigned)p.block_size), 7);
    p.box = 1 << p.box_shift;
    std::vector<std::pair<int64_t, int64_t>> lens;
    for (int i = 7; i < argc; ++i) {
        char* rest;
        const int64_t seq = std::strtoll(argv[i], &rest, 10);
        lens.emplace_back(seq, std::strtoll(rest + 1, nullptr, 10));
    }
    std::vector<int32_t> start(1, 0), seq;
    for (auto& l : lens) {
        start.push_back(start.back() + (int32_t)l.second);
        seq.push_back((int32_t)l.first);
    }
    p.B = (int)lens.size();
    p.T = start.back();
    p.q_start = start.data();
    p.seq = seq.data();
    // (zeros of which only the pages that are read take memory)
    const size_t entries = (size_t)p.B * p.max_blocks;
    p.tables = static_cast<int32_t*>(std::calloc(entries, sizeof(int32_t)));
    if (!p.tables) fail("no memory");
    unsigned status[64] = {};
    p.ctrl = status;
    readable = {{start.data(), start.size()}, {seq.data(), seq.size()}, {p.tables, entries}};
    check<Few>(p, lens);
    check<Many>(p, lens);
    return 0;
}
