// Where the padding rows begin, run by a host compiler:
//   attn_padding_host T q_start ...
#define main host_main
#include "attn_work_host.cpp"
#undef main

int main(int argc, char** argv) {
    AttnParams p = {};
    p.T = std::atoi(argv[1]);
    std::vector<int32_t> start;
    for (int i = 2; i < argc; ++i) start.push_back(std::atoi(argv[i]));
    p.B = (int)start.size() - 1;
    p.q_start = start.data();
    readable = {{start.data(), start.size()}};
    std::printf("%d\n", attn_padding(p));
    return 0;
}
