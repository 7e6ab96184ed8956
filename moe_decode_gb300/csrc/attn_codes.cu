// Attention over a paged cache of e4m3 codes with a power of two for each token
// and head: decoding streams, verify chains and trees, and (32 rows at a time)
// any other request.
//
// With codes c, exponents e and the powers of two apart, a row's score of key j
// is x_j = log2(e) scale (q . ck_j) 2^ek_j, and its output
//   o = sum_j 2^(x_j - m) 2^ev_j cv_j / sum_j 2^(x_j - m).
// A code is exact in fp16, and so is a query times a power of two of its row's
// own (bf16 has fewer bits; what lies 2^28 below the row's largest is rounded),
// so both products run on fp16 operands with fp32 sums, whatever the queries'
// type. The second one's weights are 2^(x_j + ev_j - w) with a reference w of
// their own, by the largest x + ev of the row: rounded once to fp16, they keep
// their 11 bits however the values' exponents differ.
#include <type_traits>

#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kRows = kAttnRows;
constexpr int kConsumers = 8;
constexpr int kThreads = 384;  // two warpgroups of consumers, one of producers
constexpr int kLoaders = 3;    // warps that bring tiles, in turn; a fourth brings queries
// Sums of 32 rows of 128 dimensions are 128 registers of a thread: the consumers
// take registers from the third warpgroup. Together exactly what the block is
// launched with.
constexpr int kLaunchRegs = 168, kConsumerRegs = 232, kProducerRegs = 40;
static_assert(2 * kConsumerRegs + kProducerRegs == 3 * kLaunchRegs, "registers of the block");
constexpr int kWarpKeys = kAttnTile / kConsumers;  // 16
static_assert(kWarpKeys == 16, "one step of the second product");

// A weight is at most 2^15, the least that is held 2^-24: 2^-35 of the largest
// when that has just become the reference, and 2^-39 before the next.
constexpr float kBias = 11.f, kLimit = 15.f;
// A reference before the first key: below any score, and finite, so that a score
// of -inf has the weight 0 by it.
constexpr float kNone = -3e38f;

template <int D>
struct CodesShape {
    static constexpr int kHalf = kAttnTile * D;  // K (or V) of a tile
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kQRow = D * 2 + 16;  // eight rows' 16-byte pieces in different banks
    static constexpr int kQ = kRows * kQRow;  // queries of an item, of two in turn
    static constexpr int kMerge = kRows * D * 4;
    static constexpr int kOffScale = kStages * kStage;  // of a stage: the bytes of K, then of V
    static constexpr int kOffQ = kOffScale + kStages * 2 * kAttnTile;
    static constexpr int kOffMerge = kOffQ + 2 * kQ;
    static constexpr int kOffStat = kOffMerge + kMerge;  // largest score and sum of each warp's rows
    static constexpr int kOffRow = kOffStat + (kConsumers + 1) * kRows * 8;  // powers of two of the queries
    static constexpr int kOffBar = kOffRow + kRows * 4;
    static constexpr int kOffMisc = kOffBar + 16 * (kStages + 2);
    static constexpr int kBytes = kOffMisc + 8 * (kThreads / 32) + (int)sizeof(Start) + 16 + 4 * kLoaders + 4;
    static_assert(kBytes <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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
// The transpose of an 8 x 8 tile of 16-bit elements: thread l gives row l / 4,
// elements 2 (l % 4) and 2 (l % 4) + 1, and receives those of the transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}
// One box of a cache's tensor map (dimensions, token of the block, head, block):
// `box` keys, D bytes a key in the swizzle of that width.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int token, int head, int block, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(0), "r"(token), "r"(head), "r"(block), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 16 bytes by the thread itself; copies_arrive then counts for the barrier once
// all its copies are there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A key's power of two from its byte, times 2^-less (the queries' factors make up
// for it, so that neither the sums of a row's products nor their products with
// this pass fp32's range); a value's exponent. 255 is NaN.
constexpr int kLess = 24;
__device__ __forceinline__ float key_power(uint32_t byte, int less) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : (uint32_t)max((int)byte - less, 0) << 23);
}
// A row's factor of its scores from its queries' power of two.
__device__ __forceinline__ float row_factor(const AttnParams& p, int s, int less) {
    return exp2i(-s) * (p.scale_log2 * exp2i(less));
}
__device__ __forceinline__ float value_exponent(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : (float)((int)byte - 127);
}

// The 16-byte piece c of a key's row in a tile.
template <int D>
__device__ __forceinline__ int piece_at(int key, int c) {
    return D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
}

// A row's statistics by the reference at which its sum of weights lies in [1/2, 1):
// what is scaled to that, sums of weights times values, then lies near the output,
// and passes fp32's range only where that does. (The reference is rounded, and the
// sum goes by the reference as it is.)
__device__ __forceinline__ float2 row_total(float m, float sum) {
    const float ref = m + (float)((int)(__float_as_uint(sum) >> 23) - 126);
    return make_float2(ref, sum * exp2_approx(m - ref));
}

// Joins the parts of an item, in the order of the keys (the part 1 of the CTA
// that it begins in, then the part 0 of the CTAs after it), all consumers
// together: the parts' statistics come at once, then the rows, 4 dimensions a
// thread, several parts' loads in flight. `stat`: place for kRows values.
template <int D, int DT>
__device__ __forceinline__ void join_parts(const AttnParams& p, const Span& span, int rows, int row0, int head, int token0,
                                           float2* stat, int tid) {
    constexpr int kFloats = attn_part_floats(kRows, D), kPer = D / 4, kNum = kConsumers * 32;
    const float* first = p.part + ((int64_t)span.cta * 2 + 1) * kFloats;
    const float* rest = p.part + (int64_t)span.cta * 2 * kFloats;  // part 0 of the k-th CTA at k * 2 * kFloats
    auto part_of = [&](int k) { return k == 0 ? first : rest + (int64_t)k * 2 * kFloats; };
    {
        // eight threads a row; whole warps at the shuffles, so those past the
        // last row take it again
        static_assert(kNum == 8 * kRows, "every row at once");
        const int row = min(tid / 8, rows - 1);
        auto stat_of = [&](int k) { return __ldcg(reinterpret_cast<const float2*>(part_of(k) + kRows * D) + row); };
        float mx = kNone, sum = 0.f;
        for (int k = tid % 8; k < span.parts; k += 8) mx = fmaxf(mx, stat_of(k).x);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        for (int k = tid % 8; k < span.parts; k += 8) sum += stat_of(k).y * exp2_approx(stat_of(k).x - mx);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (tid % 8 == 0 && tid / 8 < rows) stat[row] = row_total(mx, sum);
    }
    warps_sync(1, kNum);
    for (int i = tid; i < rows * kPer; i += kNum) {
        const int row = i / kPer;
        const float2 all = stat[row];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = 0; k < span.parts; ++k) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part_of(k)) + i);
            const float f = exp2_approx(__ldcg(reinterpret_cast<const float2*>(part_of(k) + kRows * D) + row).x - all.x);
            v.x += f * x.x; v.y += f * x.y; v.z += f * x.z; v.w += f * x.w;
        }
        const float inv = all.y != 0.f ? 1.f / all.y : 0.f;
        const int R = row0 + row, t = token_of(p, R), h = head * p.group + (R - t * p.group);
        const int64_t at_row = (int64_t)(token0 + t) * p.heads + h;
        *reinterpret_cast<uint2*>(p.out + at_row * D + (i % kPer) * 4) = make_uint2(pack2<DT>(v.x * inv, v.y * inv), pack2<DT>(v.z * inv, v.w * inv));
        if (i % kPer == 0 && p.lse) p.lse[at_row] = all.y != 0.f ? (all.x + log2f(all.y)) * kLn2 : -INFINITY;
    }
}

// Eight consumer warps share a tile's 128 keys, 16 each, so that a code is
// turned into fp16 once for all of the item's 32 rows; they are joined at the
// end of the item. Codes are the 16-row operand of both products and the queries
// the one of 8 columns (S^T = K Q^T, O^T = V^T P^T): an item of 8 rows takes half
// the matrix instructions that 16 rows of queries would, one of 24 three
// quarters of those of 32. Codes come out of shared memory four at a time: of K
// the four dimensions 4i..4i+3 of a key, which the queries' order in shared memory
// answers; of V two dimensions of two keys, whose even and odd dimensions are the
// product's rows i and i + 8. Three loading warps keep the ring of tiles filled
// (160 KB on their way), a fourth brings the next item's queries.
//
// 4 streams of 120,000 to 131,000 keys (64/8 heads of 128, 8 rows an item) take
// 174 to 198 us replayed from a graph, 5.2 to 5.9 TB/s; the 16-bit cache takes
// 310. 32 streams of 6 new tokens over 300 to 16,000 keys (24 rows, pages of 16)
// take 142 us (174), of 8 tokens (32 rows) 182 (176), bound by fetching and
// issuing the instructions of two warps a scheduler: 2,150 cycles a tile of 24
// rows, where HBM would take 1,470 and the matrix unit is busy for 770. One token
// over 1,001 keys takes 12.3 us (11.6): latency.
template <int D, int DT, bool TREE>
__global__ __launch_bounds__(kThreads, 1) void attn_codes_kernel(const __grid_constant__ AttnParams p,
                                                                  const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap) {
    using S = CodesShape<D>;
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
    volatile int* loaded = join_info + 3;       // the last tile that each loader has issued
    volatile int* less = loaded + kLoaders;     // key_power's, for the item at hand
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full + 8 * s, 1 + 32);  // boxes, and each lane's powers of two
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
    const Place at = attn_place<All, kThreads>(p, blockIdx.x, scan, found);
    // padding rows
    for (int64_t i = (int64_t)attn_padding(p) * p.heads + blockIdx.x + (int64_t)p.G * warp;
         i < (int64_t)p.T * p.heads; i += (int64_t)p.G * (kThreads / 32)) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x) reinterpret_cast<uint32_t*>(p.out + i * D)[32 * x + lane] = 0u;
        if (p.lse && lane == 0) p.lse[i] = -INFINITY;
    }
    if (at.begin >= at.end) return;
    volatile int* flag = &abort_flag;

    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (warp == kConsumers + kLoaders) {
            // the items' queries, a row a lane
            uint32_t items = 0;
            for (Walk<All> walk(p, at); walk.next(); walk.done(), ++items) {
                const uint32_t i = items & 1u;
                if (!__all_sync(0xffffffffu, attn_wait(q_empty + 8 * i, ((items >> 1) & 1u) ^ 1u, p, flag))) break;
                if (lane == 0) mbar_arrive_expect_tx(q_full + 8 * i, (uint32_t)(walk.rows * D * 2));
                __syncwarp();
                if (lane < walk.rows) {
                    const int R = walk.row0 + lane, t = token_of(p, R), h = walk.head * p.group + (R - t * p.group);
                    copy_bytes(base + S::kOffQ + i * S::kQ + lane * S::kQRow,
                               p.q + (int64_t)(walk.q.q0 + t) * p.q_token + h * p.q_head, D * 2, q_full + 8 * i);
                }
            }
            // the last copies, in flight where a consumer gave up
            if (lane == 0)
                for (uint32_t i = items > 2 ? items - 2 : 0; i < items; ++i) attn_drain(q_full + 8 * (i & 1u), (i >> 1) & 1u);
            return;
        }
        // Every kLoaders-th tile of the range: lane i brings the tile's i-th box,
        // if a row sees any of it. (With one warp for all, whose 16 keys a box
        // were behind the consumers, heads of 64 took 357 us for 254.)
        TileFeed<All> feed(p, at, lane);
        bool more = feed.any;
        int tile = warp - kConsumers, last = -1;
        for (int i = 0; more && i < tile; ++i) more = feed.advance();
        auto cur = feed.box(), next = cur;
        for (; more; cur = next) {
            for (int i = 0; more && i < kLoaders; ++i) more = feed.advance();
            if (more) next = feed.box();
            const int stage = tile % S::kStages;
            const uint32_t bar = full + 8 * stage;
            if (!__all_sync(0xffffffffu, attn_wait(empty + 8 * stage, ((tile / S::kStages) & 1) ^ 1, p, flag))) break;
            const bool held = p.hold_back && tile == 0;
            const bool take = attn_take(p, cur.wanted, cur.block) && !held;
            const int n = __popc(__ballot_sync(0xffffffffu, take));
            if (lane == 0 && !held) mbar_arrive_expect_tx(bar, (uint32_t)(n * p.box * 2 * D));
            __syncwarp();
            if (take) {
                const uint32_t dst = base + stage * S::kStage + lane * p.box * D;
                copy_box(dst, &kmap, cur.token, cur.head, cur.block, bar);
                copy_box(dst + S::kHalf, &vmap, cur.token, cur.head, cur.block, bar);
            }
            // The powers of two, 16 keys a lane: of K by the first 8 lanes, of V
            // by the next. (By bulk copies, four for each box of a page of 16, 32
            // requests of 6 tokens took 232 us for 188.)
            const int from = (lane & 7) << 4 >> p.box_shift;  // the lane that brings their box
            const bool there = __shfl_sync(0xffffffffu, (int)take, from) && lane < 16;
            const int block = __shfl_sync(0xffffffffu, cur.block, from), token = __shfl_sync(0xffffffffu, cur.token, from);
            if (there) {
                const int64_t byte = ((int64_t)block * p.kv_heads + cur.head) * p.block_size + token + (((lane & 7) << 4) & (p.box - 1));
                copy16(base + S::kOffScale + stage * 2 * kAttnTile + lane * 16, p.scales[lane >> 3] + byte);
            }
            copies_arrive(bar);
            last = tile;
            tile += kLoaders;
        }
        // The last copies of each stage, in flight where a consumer gave up: known
        // once no loader issues any more (a parity says nothing of a copy that
        // another has followed in its place).
        if (lane == 0) loaded[warp - kConsumers] = last;
        warps_sync(2, kLoaders * 32);
        if (warp == kConsumers && lane == 0)
            for (int s = 0; s < S::kStages; ++s) {
                int newest = -1;
                for (int i = 0; i < kLoaders; ++i)
                    for (int t = loaded[i]; t > newest; t -= kLoaders)
                        if (t % S::kStages == s) newest = t;
                if (newest > 0 || (newest == 0 && !p.hold_back)) attn_drain(full + 8 * s, (uint32_t)((newest / S::kStages) & 1));
            }
        return;
    }

    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
    Walk<All> walk(p, at);
    const int quad = lane >> 2, pair = lane & 3;
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
    float2* stat = reinterpret_cast<float2*>(sm + S::kOffStat);  // [warp][row]
    float2* total = stat + kConsumers * kRows;                   // [row]
    const float* row_scale = reinterpret_cast<const float*>(sm + S::kOffRow);
    // [row][D], groups of 8 columns swizzled by the pair of rows
    float* merge = reinterpret_cast<float*>(sm + S::kOffMerge);
    auto merged = [&](int row, int group) { return merge + row * D + ((group ^ ((row >> 1) & 3)) << 3); };

    // The item at hand, of 8 (NT - 1) + 1 to 8 NT rows: its tiles, and its sums
    // joined in shared memory.
    auto item = [&](auto sets) {
        constexpr int NT = decltype(sets)::value;
        constexpr bool kHold = NT <= 2;  // the queries stay in registers
        const uint32_t q_addr = base + S::kOffQ + (items & 1u) * S::kQ + (lane & 7) * S::kQRow + (lane >> 3) * 16;
        uint32_t q[kHold ? NT : 1][D / 32][4];
        if (kHold)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < D / 32; ++c) ldsm_x4(q_addr + n * 8 * S::kQRow + c * 64, q[n][c]);
        const AllKeys all = attn_all_keys(walk, 0, walk.rows);
        const Tree tree = attn_tree<TREE>(walk);
        // sums of this thread's rows 8 n + 2 pair + (j & 1), dimensions 16 g +
        // 2 quad + (j >> 1); references of the scores and of the products'
        // weights, sums of weights (of this thread's keys)
        float o[NT][D / 16][4];
        float m[NT][2], w[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                m[n][r] = w[n][r] = kNone;
                l[n][r] = 0.f;
            }
#pragma unroll
            for (int g = 0; g < D / 16; ++g)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][g][j] = 0.f;
        }
        // Scores of 16 keys (rows of the product) and 8 queries each, in two sums
        // of every other step where there are few of them: a product waits for
        // the one before it.
        constexpr int kSums = NT <= 2 ? 2 : 1;
        struct Scores {
            float s[kSums][NT][4];
            int key0, stage;
            bool needed;
        };
        auto product = [&](int t, int at_stage) {
            Scores x;
            x.key0 = (walk.tile0 + t) * kAttnTile + warp * kWarpKeys;
            x.stage = at_stage;
            x.needed = attn_needs(walk, x.key0, kWarpKeys);
#pragma unroll
            for (int h = 0; h < kSums; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x.s[h][n][j] = 0.f;
            if (!x.needed) return x;
            const uint32_t ks = base + at_stage * S::kStage;
            const int k_row = warp * kWarpKeys + (lane & 7) + ((lane >> 4) << 3), k_piece = (lane >> 3) & 1;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t codes[4], b[kHold ? 1 : NT][4];
                ldsm_x4(ks + piece_at<D>(k_row, 2 * c + k_piece), codes);
                if (!kHold)
#pragma unroll
                    for (int n = 0; n < NT; ++n) ldsm_x4(q_addr + n * 8 * S::kQRow + c * 64, b[kHold ? 0 : n]);
                // codes of keys 0-7: dimensions 32 c .., 32 c + 16 ..; then of
                // keys 8-15
                uint32_t a[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    e4m3x4_to_f16x2(codes[k], a[k][0], a[k][2]);
                    e4m3x4_to_f16x2(codes[2 + k], a[k][1], a[k][3]);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(x.s[k % kSums][n], a[k], kHold ? q[kHold ? n : 0][c][2 * k] : b[kHold ? 0 : n][2 * k],
                                kHold ? q[kHold ? n : 0][c][2 * k + 1] : b[kHold ? 0 : n][2 * k + 1]);
            }
            return x;
        };
        // What a tile's scores are for: weights, sums, the second product.
        auto finish = [&](Scores& x) {
            auto& s = x.s[0];
            const int key0 = x.key0;
            const bool ragged = attn_ragged(walk, key0, kWarpKeys);
            // powers of two of this thread's keys, quad and quad + 8
            const uint8_t* bytes = sm + S::kOffScale + x.stage * 2 * kAttnTile + warp * kWarpKeys + quad;
            const int item_less = *less;
            float kf[2], ve[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                kf[k] = key_power(bytes[8 * k], item_less);
                ve[k] = value_exponent(bytes[kAttnTile + 8 * k]);
            }
            if (ragged) {
                // values that no row sees may be anything: a weight of 0 times NaN
                // is not 0, so they are cleared, and their exponents
                const int key = key0 + (lane & 15);
                if (key < walk.lo || key >= walk.hi) {
                    uint8_t* v = sm + x.stage * S::kStage + S::kHalf + (warp * kWarpKeys + (lane & 15)) * D + (lane >> 4) * (D / 2);
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (key0 + 8 * k + quad < walk.lo || key0 + 8 * k + quad >= walk.hi) ve[k] = 0.f;
                __syncwarp();
            }
            // element j is key quad + 8 (j >> 1), row j & 1; its score, in units of
            // log2, is it times the row's factor
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[n][j] = (kSums > 1 ? s[n][j] + x.s[kSums - 1][n][j] : s[n][j]) * kf[j >> 1];
            if (all.lacks(key0, kWarpKeys) || (TREE && tree.reaches(key0, kWarpKeys)))
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const RowKeys sees = attn_row_keys(walk, n * 8 + 2 * pair + r);
                        const unsigned long long mask = TREE ? attn_tree_mask(walk, tree, n * 8 + 2 * pair + r) : ~0ull;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int key = key0 + 8 * k + quad;
                            if (key > sees.last || key < sees.from || (TREE && attn_tree_hides(tree, mask, key)))
                                s[n][2 * k + r] = -INFINITY;
                        }
                    }
            // exponents of the weights, by the references as they are
            float xm[NT][4], xv[NT][4], factor[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 f = *reinterpret_cast<const float2*>(row_scale + n * 8 + 2 * pair);
                factor[n][0] = f.x;
                factor[n][1] = f.y;
            }
            bool grows = false;
            auto exponents = [&] {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        xm[n][j] = fmaf(s[n][j], factor[n][j & 1], -m[n][j & 1]);
                        xv[n][j] = fmaf(s[n][j], factor[n][j & 1], ve[j >> 1] - w[n][j & 1]);
                    }
            };
            exponents();
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) grows |= fmaxf(xm[n][j], xv[n][j]) > kLimit;
            // (rare: a row's largest score so far moves up by more than 2^4 a few
            // times, however long the row)
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float x0 = s[n][r] * factor[n][r], x1 = s[n][2 + r] * factor[n][r];
                        float big = fmaxf(x0, x1), big_v = fmaxf(x0 + ve[0], x1 + ve[1]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
                            big_v = fmaxf(big_v, __shfl_xor_sync(0xffffffffu, big_v, d));
                        }
                        if (big > m[n][r] + kLimit) {
                            l[n][r] *= exp2_approx(m[n][r] - (big - kBias));
                            m[n][r] = big - kBias;
                        }
                        const bool up = big_v > w[n][r] + kLimit;
                        const float f = up ? exp2_approx(w[n][r] - (big_v - kBias)) : 1.f;
                        if (up) w[n][r] = big_v - kBias;
#pragma unroll
                        for (int g = 0; g < D / 16; ++g) {
                            o[n][g][r] *= f;
                            o[n][g][2 + r] *= f;
                        }
                    }
                exponents();
            }
            uint32_t pb[NT][2];  // weights of keys 0-7 and 8-15, keys along the registers
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int r = 0; r < 2; ++r) l[n][r] += exp2_approx(xm[n][r]) + exp2_approx(xm[n][2 + r]);
                pb[n][0] = transpose8(f32x2_to_f16x2(exp2_approx(xv[n][0]), exp2_approx(xv[n][1])));
                pb[n][1] = transpose8(f32x2_to_f16x2(exp2_approx(xv[n][2]), exp2_approx(xv[n][3])));
            }
            const uint32_t vs = base + x.stage * S::kStage + S::kHalf;
            const int v_row = warp * kWarpKeys + (lane & 15), v_piece = lane >> 4;
            uint32_t codes[D / 32][4];
#pragma unroll
            for (int c = 0; c < D / 32; ++c) ldsm_x4_trans(vs + piece_at<D>(v_row, 2 * c + v_piece), codes[c]);
            // two keys' codes of dimensions 2i and 2i + 1: of 16 dimensions keys
            // 0-7 and 8-15, then of the next 16
#pragma unroll
            for (int g = 0; g < D / 16; ++g) {
                uint32_t a[4];  // even dimensions, odd ones; then of the later keys
                e4m3x4_to_f16x2(__byte_perm(codes[g / 2][2 * (g & 1)], 0, 0x3120), a[0], a[1]);
                e4m3x4_to_f16x2(__byte_perm(codes[g / 2][2 * (g & 1) + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(o[n][g], a, pb[n][0], pb[n][1]);
            }
            if (ragged) fence_proxy_async_shared();
        };
        // (Scores of the next tile computed ahead, two tiles at a time, and the two
        // warps of a scheduler taking turns at the products all took more time, at
        // any number of rows: what bounds the loop beside HBM is the rate at which
        // two warps a scheduler fetch and issue its instructions.)
        for (int t = walk.t0; t < walk.t1; ++t) {
            if (!wait(full + 8 * stage, parity)) break;
            Scores x = product(t, stage);
            if (x.needed) finish(x);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            if (++stage == S::kStages) {
                stage = 0;
                parity ^= 1u;
            }
        }
        // join the warps: each scales to the largest score of all, then they add
        // up, in each of eight rounds each warp an eighth of the dimensions (or
        // rows) that no other is at
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], d);
                if (quad == 0) stat[warp * kRows + n * 8 + 2 * pair + r] = make_float2(m[n][r], l[n][r]);
            }
        warps_sync(1, kConsumers * 32);
        {
            // (eight threads a row; rows past the item's last give anything. Code
            // that runs once an item comes from beyond the instruction cache: it
            // is kept short.)
            const float2 own = stat[(tid & 7) * kRows + (tid >> 3)];
            float mx = own.x;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            float sum = own.y * exp2_approx(own.x - mx);
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if ((tid & 7) == 0) total[tid >> 3] = row_total(mx, sum);
        }
        warps_sync(1, kConsumers * 32);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // (half the way at a time: with the smallest and the largest values
                // the whole is beyond fp32. Nothing was seen: 0 times infinity is
                // not 0)
                const float f = w[n][r] == kNone ? 1.f : exp2_approx(0.5f * (w[n][r] - total[n * 8 + 2 * pair + r].x));
#pragma unroll
                for (int g = 0; g < D / 16; ++g) {
                    o[n][g][r] = o[n][g][r] * f * f;
                    o[n][g][2 + r] = o[n][g][2 + r] * f * f;
                }
            }
#pragma unroll 1
        for (int x = 0; x < kConsumers; ++x) {
            auto slice = [&](auto which) {
                constexpr int e = decltype(which)::value;
                constexpr bool kHalves = D == 64;  // of the rows, by their low bit
                constexpr int g = kHalves ? e >> 1 : e;
                if ((warp ^ x) != e) return;
                // row 2 pair, and from it the others at fixed distances
                float* at = merge + 2 * pair * D + (((2 * g + (quad >> 2)) ^ pair) << 3) + 2 * (quad & 3);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (kHalves && r != (e & 1)) continue;
                        float2* to = reinterpret_cast<float2*>(at + (n * 8 + r) * D);
                        const float2 u = x > 0 ? *to : make_float2(0.f, 0.f);
                        *to = make_float2(u.x + o[n][g][r], u.y + o[n][g][2 + r]);
                    }
            };
            slice(std::integral_constant<int, 0>{});
            slice(std::integral_constant<int, 1>{});
            slice(std::integral_constant<int, 2>{});
            slice(std::integral_constant<int, 3>{});
            slice(std::integral_constant<int, 4>{});
            slice(std::integral_constant<int, 5>{});
            slice(std::integral_constant<int, 6>{});
            slice(std::integral_constant<int, 7>{});
            warps_sync(1, kConsumers * 32);
        }
    };

    for (; walk.next(); walk.done()) {
        const int q_off = S::kOffQ + (items & 1u) * S::kQ;
        wait(q_full + 8 * (items & 1u), (items >> 1) & 1u);
        // The queries in place into fp16 times a power of two that brings the
        // row's largest into [2^14, 2^15), four rows a warp. Of 16 dimensions
        // 4i, 4i+1 go to places 2i, 2i+1 and 4i+2, 4i+3 to 8+2i, 9+2i. (Rows past
        // the item's last hold anything; a row's results depend on no other.)
        // Where a row's queries are so large that its factor passes fp32's range,
        // the item takes the keys' powers of two as they are: then no factor of
        // bf16 or fp16 queries does, by scales up to 2^12. (In a register of its
        // own for the length of the item that choice costs items of 32 rows 4%.)
        constexpr int kOwn = kRows / kConsumers;
        float* factors = reinterpret_cast<float*>(sm + S::kOffRow) + warp * kOwn;
        int shift[kOwn];
        bool far = false;
#pragma unroll
        for (int r = 0; r < kOwn; ++r) {
            const int row = warp * kOwn + r;
            if (row >= walk.rows) break;
            constexpr int kWords = D / 64;  // of two dimensions a lane
            uint32_t* words = reinterpret_cast<uint32_t*>(sm + q_off + row * S::kQRow);
            float2 v[kWords];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t x = words[lane * kWords + i];
                v[i] = DT == 0 ? make_float2(bf16lo(x), bf16hi(x)) : f16x2_to_f32(x);
                top = max(top, max(__float_as_uint(v[i].x) & 0x7fffffffu, __float_as_uint(v[i].y) & 0x7fffffffu));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int s = top ? max(-113, min(126, 14 - ((int)(top >> 23) - 127))) : 0;
            const float by = exp2i(s);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const int g = lane * kWords + i, in = g & 7;  // pair of dimensions, in its group of 16
                words[(g & ~7) + (in & 1) * 4 + (in >> 1)] = f32x2_to_f16x2(v[i].x * by, v[i].y * by);
            }
            shift[r] = s;
            const float factor = row_factor(p, s, kLess);
            far |= factor > 3e38f;
            if (lane == 0) factors[r] = fmaxf(factor, 1e-45f);  // (0 times a score of -inf is not that)
        }
        far = warps_any(1, kConsumers * 32, far);
        if (tid == 0) *less = far ? 0 : kLess;
        if (far) {
            if (lane == 0)
#pragma unroll
                for (int r = 0; r < kOwn; ++r)
                    if (warp * kOwn + r < walk.rows) factors[r] = fminf(fmaxf(row_factor(p, shift[r], 0), 1e-45f), 3e38f);
        }
        warps_sync(1, kConsumers * 32);
        if (walk.rows <= 8) item(std::integral_constant<int, 1>{});
        else if (walk.rows <= 16) item(std::integral_constant<int, 2>{});
        else if (walk.rows <= 24) item(std::integral_constant<int, 3>{});
        else item(std::integral_constant<int, 4>{});
        // (this warp's rows of the queries were written in place: the next copy
        // into them comes after)
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + 8 * (items & 1u));
        ++items;
        // 16 bytes of output a thread
        const bool whole = walk.whole();
        float* part = p.part + ((int64_t)blockIdx.x * 2 + walk.part()) * attn_part_floats(kRows, D);
#pragma unroll 1
        for (int i = tid; i < walk.rows * (D / 8); i += kConsumers * 32) {
            const int row = i / (D / 8), c = i % (D / 8);
            const float4* sum = reinterpret_cast<const float4*>(merged(row, c));
            const float4 x = sum[0], y = sum[1];
            if (whole) {
                const float2 ml = total[row];
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
                if (c == 0) reinterpret_cast<float2*>(part + kRows * D)[row] = total[row];
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
                join_parts<D, DT>(p, Span{join_info[0], join_info[1]}, walk.rows, walk.row0, walk.head, walk.q.q0, total, tid);
            warps_sync(1, kConsumers * 32);
        }
    }
}

template <int D, int DT, bool TREE>
cudaError_t launch_typed(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    auto* kern = attn_codes_kernel<D, DT, TREE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, CodesShape<D>::kBytes);
    if (e != cudaSuccess) return e;
    // the warpgroups' shares wait for ever where the launch brings fewer
    cudaFuncAttributes have;
    e = cudaFuncGetAttributes(&have, kern);
    if (e != cudaSuccess) return e;
    if (have.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.G);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = CodesShape<D>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, k, v);
}

template <int D, int DT>
cudaError_t launch_tree(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    return p.tree ? launch_typed<D, DT, true>(p, k, v, stream) : launch_typed<D, DT, false>(p, k, v, stream);
}

}  // namespace

cudaError_t launch_attn_codes(const AttnParams& p, const void* k_map, const void* v_map, int head_dim, int dtype,
                              cudaStream_t stream) {
    const CUtensorMap& k = *static_cast<const CUtensorMap*>(k_map);
    const CUtensorMap& v = *static_cast<const CUtensorMap*>(v_map);
    if (head_dim == 128) return dtype == 0 ? launch_tree<128, 0>(p, k, v, stream) : launch_tree<128, 1>(p, k, v, stream);
    return dtype == 0 ? launch_tree<64, 0>(p, k, v, stream) : launch_tree<64, 1>(p, k, v, stream);
}

}  // namespace moe
