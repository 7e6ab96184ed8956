// The checks of attn_work_host.cpp for the divisions of the work of attention
// over a cache of 8-bit values (every request in items of 32 rows) and of calls
// with trees. The same arguments.
#define main host_main
#include "attn_work_host.cpp"
#undef main

// The CTAs that have tiles of an item are as many as its count says, one after
// another from its first.
template <class Class>
static void parts(const AttnParams& p) {
    Place at = {};
    for (int r = 0; r < p.B; ++r) {
        const Request q = attn_request(p, r);
        if (Class::mine(p, q)) at.total += attn_request_units<Class>(p, q) * p.kv_heads;
    }
    std::map<std::tuple<int, int, int>, std::pair<int, int>> at_item;  // CTAs so far, their count
    for (int cta = 0; cta < p.G; ++cta) {
        attn_range(p, cta, at);
        if (at.begin >= at.end) continue;
        at.start = attn_seek<Class>(p, 0, p.B, at.begin);
        for (Walk<Class> w(p, at); w.next(); w.done()) {
            const Span s = attn_span(w, at);
            auto& have = at_item[{w.r, w.head, w.row0}];
            if (cta != s.cta + have.first) fail("a CTA between without a tile");
            ++have.first;
            have.second = s.parts;
        }
    }
    for (const auto& i : at_item)
        if (i.second.first != i.second.second) fail("a count of parts that is not that of the CTAs");
}

int main(int argc, char** argv) {
    if (host_main(argc, argv)) return 1;
    AttnParams p = {};
    int32_t* number[] = {&p.block_size, &p.window, &p.max_blocks, &p.kv_heads, &p.group, &p.G};
    for (int i = 0; i < 6; ++i) *number[i] = std::atoi(argv[1 + i]);
    p.heads = p.kv_heads * p.group;
    p.group_magic = ((1ull << 36) + p.group - 1) / p.group;
    p.box_shift = std::min(__builtin_ctz((unsigned)p.block_size), 7);
    p.box = 1 << p.box_shift;
    std::vector<std::pair<int64_t, int64_t>> lens;
    std::vector<int32_t> start(1, 0), seq;
    for (int i = 7; i < argc; ++i) {
        char* rest;
        const int64_t n = std::strtoll(argv[i], &rest, 10);
        lens.emplace_back(n, std::strtoll(rest + 1, nullptr, 10));
        start.push_back(start.back() + (int32_t)lens.back().second);
        seq.push_back((int32_t)n);
    }
    p.B = (int)lens.size();
    p.T = start.back();
    p.q_start = start.data();
    p.seq = seq.data();
    const size_t entries = (size_t)p.B * p.max_blocks;
    p.tables = static_cast<int32_t*>(std::calloc(entries, sizeof(int32_t)));
    if (!p.tables) fail("no memory");
    unsigned status[64] = {};
    p.ctrl = status;
    readable = {{start.data(), start.size()}, {seq.data(), seq.size()}, {p.tables, entries}};
    check<FewTree>(p, lens);
    check<ManyTree>(p, lens);
    check<All>(p, lens);
    parts<All>(p);
    parts<FewTree>(p);
    parts<ManyTree>(p);
    return 0;
}
