// The checks of attn_work_host.cpp for the divisions of the work of attention
// over a cache of 8-bit values (every request in items of 32 rows) and of calls
// with trees. The same arguments.
#define main host_main
#include "attn_work_host.cpp"
#undef main

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
    check<All>(p, lens);
    check<FewTree>(p, lens);
    check<ManyTree>(p, lens);
    return 0;
}
