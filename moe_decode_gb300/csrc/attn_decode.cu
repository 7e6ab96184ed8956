// Attention of few query rows over the paged cache: decoding streams, verify
// chains and short chunks.
#include <type_traits>

#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kRows = kAttnRows;
constexpr int kKeyWarps = 4;               // warps that share a tile's keys
constexpr int kConsumers = 2 * kKeyWarps;  // for each of two sets of 16 rows; one producer warp on top
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kWarpKeys = kAttnTile / kKeyWarps;

template <int D>
struct DecodeShape {
    static constexpr int kHalf = kAttnTile * D * 2;          // K (or V) of a tile
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kQRow = D * 2 + 16;                 // eight rows' 16-byte pieces in different banks
    static constexpr int kQ = kRows * kQRow;                 // queries of an item, of two in turn
    static constexpr int kMerge = kRows * D * 4;
    static constexpr int kOffQ = kStages * kStage;
    static constexpr int kOffMerge = kOffQ + 2 * kQ;
    static constexpr int kOffStat = kOffMerge + kMerge;      // largest score and sum of each warp's rows
    static constexpr int kOffBar = kOffStat + kKeyWarps * kRows * 8;
    static constexpr int kOffMisc = kOffBar + 16 * (kStages + 2);
    static constexpr int kBytes = kOffMisc + 8 * (kThreads / 32) + (int)sizeof(Start) + 16;
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

// One row of queries (16-byte aligned at both ends) into shared memory.
__device__ __forceinline__ void copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int DT>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (DT == 0)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Each consumer warp takes 32 keys of every tile against 16 of the item's 32
// rows, with its own running largest score, sum and output; the four warps of
// a set of rows are joined once at the end of the item. A producer warp keeps
// three tiles of 128 keys (192 KB at 128 dimensions) on their way, across
// items, and the queries of the item after the one at hand.
//
// Bound by HBM where the histories are long (times are of calls replayed from a
// graph): 4 streams of 120,000 to 131,000 keys (64/8 heads of 128) take 309 us,
// 6.7 TB/s; 32 streams of 6 new tokens over 300 to 16,000 keys (24 rows an item,
// pages of 16) 174 us, 5.9 TB/s in the kernel. Four warps with 32 rows each took 206 us there: the second set of
// warps hides the first's chains. Short histories are bound by latency: one
// token over 1,001 keys takes 11.2 us.
//
// TREE: rows see of their request's new tokens those that their masks name. Only
// the last tiles of an item look at the masks; a kernel without is compiled as
// before.
template <int D, int DT, bool TREE>
__global__ __launch_bounds__(kThreads, 1) void attn_decode_kernel(const __grid_constant__ AttnParams p,
                                                                   const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap) {
    using Class = std::conditional_t<TREE, FewTree, Few>;
    using S = DecodeShape<D>;
    // (no static shared memory: this begins on a 1024-byte boundary, which the
    // swizzle counts from)
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // barriers: key/value stages and queries, each full and empty
    const uint32_t full = base + S::kOffBar, empty = full + 8 * S::kStages;
    const uint32_t q_full = empty + 8 * S::kStages, q_empty = q_full + 16;
    int64_t* scan = reinterpret_cast<int64_t*>(sm + S::kOffMisc);
    Start* found = reinterpret_cast<Start*>(scan + kThreads / 32);
    int& abort_flag = *reinterpret_cast<int*>(found + 1);
    volatile int* join_info = &abort_flag + 1;  // first CTA, parts, whether this one is the last
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, kConsumers);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + 8 * i, 1);
            mbar_init(q_empty + 8 * i, kConsumers);
        }
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const Place at = attn_place<Class, kThreads>(p, blockIdx.x, scan, found);
    // padding rows
    for (int64_t i = (int64_t)attn_padding(p) * p.heads + blockIdx.x + (int64_t)p.G * warp;
         i < (int64_t)p.T * p.heads; i += (int64_t)p.G * (kThreads / 32)) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x) reinterpret_cast<uint32_t*>(p.out + i * D)[32 * x + lane] = 0u;
        if (p.lse && lane == 0) p.lse[i] = -INFINITY;
    }
    if (at.begin >= at.end) return;
    volatile int* flag = &abort_flag;

    if (warp == kConsumers) {
        // producer: lane i brings the tile's i-th box, if a row sees any of it
        int stage = 0, issued = 0;
        uint32_t parity = 1, items = 0;
        TileFeed<Class> feed(p, at, lane);
        auto cur = feed.box(), next = cur;
        for (bool more = feed.any; more; cur = next) {
            more = feed.advance();
            if (more) next = feed.box();
            if (cur.rows > 0) {
                // the item's queries, a row a lane
                const uint32_t i = items & 1u;
                if (!__all_sync(0xffffffffu, attn_wait(q_empty + 8 * i, ((items >> 1) & 1u) ^ 1u, p, flag))) break;
                if (lane == 0) mbar_arrive_expect_tx(q_full + 8 * i, (uint32_t)(cur.rows * D * 2));
                __syncwarp();
                if (lane < cur.rows) {
                    const int R = cur.row0 + lane, t = token_of(p, R), h = cur.head * p.group + (R - t * p.group);
                    copy_row(base + S::kOffQ + i * S::kQ + lane * S::kQRow,
                             p.q + (cur.token0 + t) * p.q_token + h * p.q_head, D * 2, q_full + 8 * i);
                }
                ++items;
            }
            if (!__all_sync(0xffffffffu, attn_wait(empty + 8 * stage, parity, p, flag))) break;
            const bool held = p.hold_back && issued == 0;
            const bool take = attn_take(p, cur.wanted, cur.block) && !held;
            const int n = __popc(__ballot_sync(0xffffffffu, take));
            if (lane == 0 && !held) mbar_arrive_expect_tx(full + 8 * stage, (uint32_t)(n * p.box * D * 4));
            __syncwarp();
            if (take) {
                const uint32_t dst = base + stage * S::kStage + lane * p.box * D * 2;
                attn_copy(dst, &kmap, 0, cur.token, cur.head, cur.block, full + 8 * stage);
                attn_copy(dst + S::kHalf, &vmap, 0, cur.token, cur.head, cur.block, full + 8 * stage);
            }
            ++issued;
            if (++stage == S::kStages) {
                stage = 0;
                parity ^= 1u;
            }
        }
        // the last copies of each stage, in flight where a consumer gave up
        if (lane == 0) {
            for (int i = max(p.hold_back, issued - S::kStages); i < issued; ++i)
                attn_drain(full + 8 * (i % S::kStages), (uint32_t)((i / S::kStages) & 1));
            for (uint32_t i = items > 2 ? items - 2 : 0; i < items; ++i) attn_drain(q_full + 8 * (i & 1u), (i >> 1) & 1u);
        }
        return;
    }

    Walk<Class> walk(p, at);
    const int quad = lane >> 2, pair = lane & 3;
    const int set = warp / kKeyWarps, kw = warp % kKeyWarps;  // rows [16 set, 16 set + 16), a quarter of the keys
    // a key's row in a stage: boxes of `box` keys, in each the panels of 64
    // dimensions one after another
    const int panel = p.box * 128;
    auto key_at = [&](int key) { return (key >> p.box_shift) * (p.box * D * 2) + (key & (p.box - 1)) * 128; };
    int k_at[2], v_at[2];  // rows that this lane names to ldmatrix, of 16 keys each
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        k_at[h] = key_at(kw * kWarpKeys + h * 16 + ((lane >> 4) << 3) + (lane & 7));
        v_at[h] = key_at(kw * kWarpKeys + h * 16 + (lane & 15));
    }
    int stage = 0;
    uint32_t parity = 0;
    uint32_t items = 0;
    // A wait that ran out ends the work of the warp, but not its way past the
    // barriers that the others stand at.
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t par) {
        ok = __all_sync(0xffffffffu, ok && attn_wait(bar, par, p, flag));
        return ok;
    };
    float2* stat = reinterpret_cast<float2*>(sm + S::kOffStat);  // [key warp][row]
    float* merge = reinterpret_cast<float*>(sm + S::kOffMerge);  // [row][D], groups of 8 columns swizzled by the row
    for (; walk.next(); walk.done()) {
        // (rows past the item's last hold anything; a row's results depend on
        // no other row)
        const uint32_t q_addr = base + S::kOffQ + (items & 1u) * S::kQ + (set * 16 + (lane & 15)) * S::kQRow + (lane >> 4) * 16;
        wait(q_full + 8 * (items & 1u), (items >> 1) & 1u);
        const bool active = set * 16 < walk.rows;
        // the last key that each of this thread's two rows sees, and the first
        int last[2], from[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const RowKeys k = attn_row_keys(walk, set * 16 + b * 8 + quad);
            last[b] = k.last;
            from[b] = k.from;
        }
        const AllKeys all = attn_all_keys(walk, 0, walk.rows);
        const Tree tree = attn_tree<TREE>(walk);
        unsigned long long mask[2] = {~0ull, ~0ull};
        if (TREE)
#pragma unroll
            for (int b = 0; b < 2; ++b) mask[b] = attn_tree_mask(walk, tree, set * 16 + b * 8 + quad);
        float o[D / 8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        for (int t = walk.t0; t < walk.t1; ++t) {
            if (!wait(full + 8 * stage, parity)) break;
            const int key0 = (walk.tile0 + t) * kAttnTile + kw * kWarpKeys;
            const uint32_t ks = base + stage * S::kStage, vs = ks + S::kHalf;
            if (active && attn_needs(walk, key0, kWarpKeys)) {
                const bool ragged = attn_ragged(walk, key0, kWarpKeys);
                if (ragged) {
                    // values that no row sees may be anything: a weight of 0 times
                    // NaN is not 0, so they are cleared (by both sets of rows,
                    // each before its own reads)
                    const int key = key0 + lane;
                    if (key < walk.lo || key >= walk.hi) {
                        uint8_t* v = sm + stage * S::kStage + S::kHalf + key_at(kw * kWarpKeys + lane);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(v + x * panel + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                float s[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t qa[4], kb[2][4];
                    ldsm_x4(q_addr + k * 32, qa);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 keys each
                        const int c = 2 * (k & 3) + ((lane >> 3) & 1);
                        ldsm_x4(ks + k_at[h] + (k >> 2) * panel + ((c ^ (lane & 7)) << 4), kb[h]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mma_16816<DT>(s[2 * h], qa, kb[h][0], kb[h][1]);
                        mma_16816<DT>(s[2 * h + 1], qa, kb[h][2], kb[h][3]);
                    }
                }
                if (all.lacks(key0, kWarpKeys)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = key0 + i * 8 + 2 * pair + (j & 1);
                            if (key > last[j >> 1] || key < from[j >> 1]) s[i][j] = -INFINITY;
                        }
                }
                if (TREE && tree.reaches(key0, kWarpKeys)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (attn_tree_hides(tree, mask[j >> 1], key0 + i * 8 + 2 * pair + (j & 1))) s[i][j] = -INFINITY;
                }
                uint32_t pa[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(s[i][2 * b], s[i][2 * b + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    mx *= p.scale_log2;
                    const bool grows = mx > m[b] + WeightRange<DT>::kLimit;
                    if (__any_sync(0xffffffffu, grows)) {
                        const float to = mx - WeightRange<DT>::kBias;
                        const float f = grows ? exp2_approx(m[b] - to) : 1.f;
                        if (grows) m[b] = to;
                        l[b] *= f;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[i][2 * b] *= f;
                            o[i][2 * b + 1] *= f;
                        }
                    }
                    const float ref = m[b] == -INFINITY ? 0.f : m[b];
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = exp2_approx(fmaf(s[i][2 * b], p.scale_log2, -ref));
                        const float y = exp2_approx(fmaf(s[i][2 * b + 1], p.scale_log2, -ref));
                        sum += x + y;
                        // rounded once to the values' type for the second
                        // product: half a step of each weight, independent
                        // from key to key; the sum keeps the fp32 weights
                        pa[i >> 1][(i & 1) * 2 + b] = pack2<DT>(x, y);
                    }
                    l[b] += sum;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        uint32_t vb[4];
                        const int c = 2 * (i & 3) + (lane >> 4);
                        ldsm_x4_trans(vs + v_at[h] + (i >> 2) * panel + ((c ^ (lane & 7)) << 4), vb);
                        mma_16816<DT>(o[2 * i], pa[h], vb[0], vb[1]);
                        mma_16816<DT>(o[2 * i + 1], pa[h], vb[2], vb[3]);
                    }
                if (ragged) fence_proxy_async_shared();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            if (++stage == S::kStages) {
                stage = 0;
                parity ^= 1u;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + 8 * (items & 1u));
        ++items;
        // join the warps that share the rows: each scales to the largest score
        // of all, then they add up one after another
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            l[b] += __shfl_xor_sync(0xffffffffu, l[b], 1);
            l[b] += __shfl_xor_sync(0xffffffffu, l[b], 2);
            if (pair == 0) stat[kw * kRows + set * 16 + b * 8 + quad] = make_float2(m[b], l[b]);
        }
        warps_sync(1, kConsumers * 32);
        float big[2], sum[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int row = set * 16 + b * 8 + quad;
            float mx = -INFINITY, tot = 0.f;
#pragma unroll
            for (int w = 0; w < kKeyWarps; ++w) mx = fmaxf(mx, stat[w * kRows + row].x);
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int w = 0; w < kKeyWarps; ++w)
                tot += stat[w * kRows + row].y * exp2_approx(stat[w * kRows + row].x - ref);
            big[b] = mx;
            sum[b] = tot;
            const float f = exp2_approx(m[b] - ref);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][2 * b] *= f;
                o[i][2 * b + 1] *= f;
            }
        }
        for (int w = 0; w < kKeyWarps; ++w) {
            if (kw == w && active) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    // (eight loads before the first store: the compiler cannot
                    // tell the swizzled addresses apart)
                    float* row = merge + (set * 16 + b * 8 + quad) * D + 2 * pair;
#pragma unroll
                    for (int i0 = 0; i0 < D / 8; i0 += 8) {
                        float2 u[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            u[i] = w > 0 ? *reinterpret_cast<const float2*>(row + ((i0 + i) ^ (quad & 3)) * 8)
                                         : make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float2*>(row + ((i0 + i) ^ (quad & 3)) * 8) =
                                make_float2(u[i].x + o[i0 + i][2 * b], u[i].y + o[i0 + i][2 * b + 1]);
                    }
                }
            }
            // (everyone has read the statistics by the first of these)
            if (w == kKeyWarps - 1 && kw == 0 && pair == 0)
#pragma unroll
                for (int b = 0; b < 2; ++b) stat[set * 16 + b * 8 + quad] = make_float2(big[b], sum[b]);
            warps_sync(1, kConsumers * 32);
        }
        // 16 bytes of output a thread
        const bool whole = walk.whole();
        float* part = p.part + ((int64_t)blockIdx.x * 2 + walk.part()) * attn_part_floats(kRows, D);
        for (int i = tid; i < walk.rows * (D / 8); i += kConsumers * 32) {
            const int row = i / (D / 8), c = i % (D / 8);
            const float4 x = *reinterpret_cast<const float4*>(merge + row * D + (c ^ (row & 3)) * 8);
            const float4 y = *reinterpret_cast<const float4*>(merge + row * D + (c ^ (row & 3)) * 8 + 4);
            if (whole) {
                const float2 ml = stat[row];
                const float inv = ml.y != 0.f ? 1.f / ml.y : 0.f;
                const int R = walk.row0 + row, t = token_of(p, R), h = walk.head * p.group + (R - t * p.group);
                const int64_t at_row = (int64_t)(walk.q.q0 + t) * p.heads + h;
                uint4 v;
                v.x = pack2<DT>(x.x * inv, x.y * inv);
                v.y = pack2<DT>(x.z * inv, x.w * inv);
                v.z = pack2<DT>(y.x * inv, y.y * inv);
                v.w = pack2<DT>(y.z * inv, y.w * inv);
                *reinterpret_cast<uint4*>(p.out + at_row * D + c * 8) = v;
                if (c == 0 && p.lse) p.lse[at_row] = ml.y != 0.f ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
            } else {
                *reinterpret_cast<float4*>(part + row * D + c * 8) = x;
                *reinterpret_cast<float4*>(part + row * D + c * 8 + 4) = y;
                if (c == 0) reinterpret_cast<float2*>(part + kRows * D)[row] = stat[row];
            }
        }
        // the next item writes the rows and the statistics after this barrier
        warps_sync(1, kConsumers * 32);
        if (!whole) {
            if (tid == 0) {
                const Span span = attn_span(walk, at);
                join_info[0] = span.cta;
                join_info[1] = span.parts;
                join_info[2] = attn_last(p.arrived + span.cta, span.parts);
            }
            warps_sync(1, kConsumers * 32);
            if (join_info[2])
                attn_join<D, DT, kRows, kConsumers * 32, 2>(p, p.part, Span{join_info[0], join_info[1]}, 0, walk.rows,
                                                         walk.row0, walk.head, walk.q.q0, tid);
            warps_sync(1, kConsumers * 32);
        }
    }
}

template <class... Args>
cudaError_t launch(void (*kern)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int D, int DT, bool TREE>
cudaError_t launch_typed(const AttnParams& p, const CUtensorMap* maps, cudaStream_t stream, int* launches) {
    cudaError_t e = launch(attn_decode_kernel<D, DT, TREE>, dim3((unsigned)p.G), kThreads, DecodeShape<D>::kBytes, stream, p,
                           maps[0], maps[1]);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (attn_may_chunk(p)) {
        e = launch_attn_chunk(p, &maps[2], &maps[3], D, DT, stream);
        if (e == cudaSuccess) ++*launches;
    }
    return e;
}

}  // namespace

cudaError_t launch_attn(const AttnParams& p, const void* maps, int head_dim, int dtype, cudaStream_t stream,
                        int* launches) {
    const CUtensorMap* m = static_cast<const CUtensorMap*>(maps);
    *launches = 0;
    if (p.tree) {
        if (head_dim == 128)
            return dtype == 0 ? launch_typed<128, 0, true>(p, m, stream, launches) : launch_typed<128, 1, true>(p, m, stream, launches);
        return dtype == 0 ? launch_typed<64, 0, true>(p, m, stream, launches) : launch_typed<64, 1, true>(p, m, stream, launches);
    }
    if (head_dim == 128)
        return dtype == 0 ? launch_typed<128, 0, false>(p, m, stream, launches) : launch_typed<128, 1, false>(p, m, stream, launches);
    return dtype == 0 ? launch_typed<64, 0, false>(p, m, stream, launches) : launch_typed<64, 1, false>(p, m, stream, launches);
}

}  // namespace moe
