// Bookkeeping of a paged KV cache for one step: block tables, slot map and
// positions from the requests' lengths (moe_paged_plan), and the write of the
// step's keys and values through the slot map (moe_paged_append).
#include "layer_params.h"
#include "paged.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 512;

__device__ __forceinline__ void report(unsigned* ctrl, int code) {
    atomicCAS(reinterpret_cast<int*>(ctrl + kCtlStatus), 0, code);
}

// Exclusive sums over the block's threads of a pair of values; tot receives
// the block's totals.
__device__ __forceinline__ void block_scan(long long& a, long long& b, long long (&tot)[2]) {
    __shared__ long long sums[2][kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sums[0][warp] = a;
        sums[1][warp] = b;
    }
    __syncthreads();
    long long pa = 0, pb = 0;
    tot[0] = tot[1] = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const long long x = sums[0][w], y = sums[1][w];
        if (w < warp) {
            pa += x;
            pb += y;
        }
        tot[0] += x;
        tot[1] += y;
    }
    a = pa + a - a0;
    b = pb + b - b0;
}

// Largest i in [0, n) with v[i] <= x (v ascending, v[0] <= x).
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Every CTA sums up all requests' tokens and missing blocks by itself (8
// bytes a request, out of L2 but for the first), so that no CTA waits for
// another; then tokens and new blocks are spread over the grid, each found in
// the prefix sums by bisection in shared memory. A token in a new block takes
// its block from the free list directly, not from the table that another CTA
// may be writing. Bound by the launch: 16 requests of 6 tokens (one CTA) take
// 4.1 us a graph-replayed call, 512 requests of 40,895 tokens (80 CTAs) 4.9.
__global__ __launch_bounds__(kPlanThreads) void paged_plan_kernel(PlanParams p) {
    __shared__ int q0[kMaxRequests + 1];     // first token of each request
    __shared__ int first[kMaxRequests + 1];  // first new block of each request
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, bs = p.block_size;
    const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    bool bad = false, over = false;
    long long toks = 0, blks = 0;
    const int row_cap = p.max_blocks;
    auto lens = [&](int b, int& c, int& n, int& have, int& need) {
        c = p.ctx[b];
        n = p.fresh[b];
        if (c < 0 || n < 0) bad = true;
        c = max(c, 0);
        n = max(n, 0);
        if (n > 0x7fffffff - c) {
            bad = true;
            n = 0x7fffffff - c;
        }
        have = (int)(((long long)c + bs - 1) / bs);
        const int want = (int)(((long long)c + n + bs - 1) / bs);
        if (n > 0 && want > row_cap) over = true;
        need = max(min(want, row_cap) - have, 0);
    };
    for (int b = b0; b < b1; ++b) {
        int c, n, have, need;
        lens(b, c, n, have, need);
        toks += n;
        blks += need;
    }
    long long tot[2];
    block_scan(toks, blks, tot);
    for (int b = b0; b < b1; ++b) {
        int c, n, have, need;
        lens(b, c, n, have, need);
        q0[b] = (int)min(toks, 0x7fffffffLL);
        first[b] = (int)min(blks, 0x7fffffffLL);
        if (blockIdx.x == 0) {
            p.q_start[b] = q0[b];
            p.seq[b] = c + n;
        }
        toks += n;
        blks += need;
    }
    const int total = (int)min(tot[0], 0x7fffffffLL), blocks = (int)min(tot[1], 0x7fffffffLL);
    int head = p.free_head ? *p.free_head : 0;
    if (head < 0) {
        bad = true;
        head = p.n_free;
    }
    const int avail = max(p.n_free - head, 0), given = min(blocks, avail);
    if (blocks > avail || total > p.T || tot[0] > total) over = true;
    if (blockIdx.x == 0 && tid == 0) {
        p.q_start[p.B] = total;
        *p.taken = given;
    }
    __syncthreads();

    const int step = gridDim.x * kPlanThreads, id = blockIdx.x * kPlanThreads + tid;
    // new blocks: the e-th goes to column have + e - first of its request
    for (int64_t e = id; e < given; e += step) {
        const int b = last_at_most(first, p.B, (int)e);
        const int have = (int)(((long long)max(p.ctx[b], 0) + bs - 1) / bs);
        p.tables[(int64_t)b * p.max_blocks + have + (e - first[b])] = p.free_list[head + e];
    }
    for (int64_t t = id; t < p.T; t += step) {
        int slot = -1, pos = -1;
        if (t < total) {
            const int b = last_at_most(q0, p.B, (int)t);
            const int c = max(p.ctx[b], 0);
            pos = c + ((int)t - q0[b]);  // (the sum of c and t may pass 32 bits)
            const int page = pos / bs, have = (int)(((long long)c + bs - 1) / bs);
            int block = -1;
            if (page < p.max_blocks) {
                if (page < have) {
                    block = p.tables[(int64_t)b * p.max_blocks + page];
                    if (block < 0) bad = true;
                } else {
                    const int64_t e = (int64_t)first[b] + (page - have);
                    if (e < given) {
                        block = p.free_list[head + e];
                        if (block < 0) bad = true;
                    }
                }
            }
            const long long s = (long long)block * bs + pos % bs;
            if (block >= 0 && s > 0x7fffffffLL) bad = true;
            if (block >= 0 && s <= 0x7fffffffLL) slot = (int)s;
        }
        p.slots[t] = slot;
        if (p.positions) p.positions[t] = pos;
    }
    if (bad) report(p.ctrl, -100 /* MOE_EDEVICE_BAD_INDEX */);
    if (over) report(p.ctrl, -102 /* MOE_EDEVICE_OVERFLOW */);
}

// One warp a token: its lanes take the token's 16-byte pieces, keys and
// values in the same round, four rounds unrolled (16 KB of a token of 8 heads
// of 128 in flight a warp). Bound by HBM: 8,192 tokens of 8 heads of 128 take
// 11.6 us, 5.4 TB/s read and written.
__global__ __launch_bounds__(256) void paged_append_kernel(AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int pieces = p.heads << p.dim_shift, mask = (1 << p.dim_shift) - 1;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < p.T; t += warps) {
        const int slot = p.slots[t];
        if (slot < 0 || slot >= p.n_slots) {
            if (slot != -1 && lane == 0) report(p.ctrl, -100 /* MOE_EDEVICE_BAD_INDEX */);
            continue;
        }
        const int block = slot / p.block_size, at = slot - block * p.block_size;
        const uint16_t* src[2];
        uint16_t* dst[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            src[i] = p.src[i] + t * p.src_token[i];
            dst[i] = p.dst[i] + block * p.dst_block[i] + at * p.dst_token[i];
        }
        for (int c0 = lane; c0 < pieces; c0 += 128) {
            uint4 v[2][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = c0 + 32 * r;
                if (c < pieces)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        v[i][r] = *reinterpret_cast<const uint4*>(src[i] + (c >> p.dim_shift) * p.src_head[i] + (c & mask) * 8);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int c = c0 + 32 * r;
                if (c < pieces)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint4*>(dst[i] + (c >> p.dim_shift) * p.dst_head[i] + (c & mask) * 8) = v[i][r];
            }
        }
    }
}

template <class P>
cudaError_t launch_pdl(void (*kern)(P), int grid, int threads, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, int sms, cudaStream_t stream) {
    const int64_t want = ((int64_t)p.T + kPlanThreads - 1) / kPlanThreads;
    const int grid = (int)(want < 1 ? 1 : want > sms ? sms : want);
    return launch_pdl(paged_plan_kernel, grid, kPlanThreads, p, stream);
}

cudaError_t launch_paged_append(const AppendParams& p, int sms, cudaStream_t stream) {
    const int64_t want = ((int64_t)p.T + 7) / 8, most = (int64_t)sms * 8;
    return launch_pdl(paged_append_kernel, (int)(want > most ? most : want), 256, p, stream);
}

}  // namespace moe
