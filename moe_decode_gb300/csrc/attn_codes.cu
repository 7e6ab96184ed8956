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
#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kRows = kAttnRows;
constexpr int kConsumers = 8;
constexpr int kThreads = 384;  // two warpgroups of consumers, one for the producer
// Sums of 32 rows of 128 dimensions are 128 registers of a thread: the consumers
// take registers from the third warpgroup. Together exactly what the block is
// launched with.
constexpr int kLaunchRegs = 168, kConsumerRegs = 224, kProducerRegs = 56;
static_assert(2 * kConsumerRegs + kProducerRegs == 3 * kLaunchRegs, "registers of the block");
constexpr int kWarpKeys = kAttnTile / kConsumers;  // 16
static_assert(kWarpKeys == 16, "one step of the second product");

// A weight is at most 2^15, the least that is held 2^-24: 2^-35 of the largest
// when that has just become the reference, and 2^-39 before the next.
constexpr float kBias = 11.f, kLimit = 15.f;

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
    static constexpr int kOffMerge = kOffQ + 2 * kQ;        // two sums of warps
    static constexpr int kOffStat = kOffMerge + 2 * kMerge;  // largest score and sum of each warp's rows
    static constexpr int kOffRow = kOffStat + kConsumers * kRows * 8;  // powers of two of the queries
    static constexpr int kOffBar = kOffRow + kRows * 4;
    static constexpr int kOffMisc = kOffBar + 16 * (kStages + 2);
    static constexpr int kBytes = kOffMisc + 8 * (kThreads / 32) + (int)sizeof(Start) + 16;
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

// The 16-byte piece c of a key's row in a tile.
template <int D>
__device__ __forceinline__ int piece_at(int key, int c) {
    return D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
}

// Eight consumer warps share a tile's 128 keys, 16 each, so that a code is
// turned into fp16 once for all of the item's 32 rows; they are joined at the
// end of the item. Codes come out of shared memory four at a time: of K the four
// dimensions 4i..4i+3 of a key, which the queries' order in shared memory
// answers; of V two dimensions of two keys, whose even and odd dimensions go to
// tiles of their own. A producer warp keeps the ring of tiles filled.
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
    const Place at = attn_place<All, kThreads>(p, blockIdx.x, scan, found);
    // padding rows
    for (int64_t i = (int64_t)min(max(p.q_start[p.B], 0), p.T) * p.heads + blockIdx.x + (int64_t)p.G * warp;
         i < (int64_t)p.T * p.heads; i += (int64_t)p.G * (kThreads / 32)) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x) reinterpret_cast<uint32_t*>(p.out + i * D)[32 * x + lane] = 0u;
        if (p.lse && lane == 0) p.lse[i] = -INFINITY;
    }
    if (at.begin >= at.end) return;
    volatile int* flag = &abort_flag;

    if (warp >= kConsumers) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
        if (warp > kConsumers) return;
        // producer: lane i brings the tile's i-th box, if a row sees any of it
        int stage = 0, issued = 0;
        uint32_t parity = 1, items = 0;
        TileFeed<All> feed(p, at, lane);
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
                    copy_bytes(base + S::kOffQ + i * S::kQ + lane * S::kQRow,
                               p.q + (cur.token0 + t) * p.q_token + h * p.q_head, D * 2, q_full + 8 * i);
                }
                ++items;
            }
            if (!__all_sync(0xffffffffu, attn_wait(empty + 8 * stage, parity, p, flag))) break;
            const bool held = p.hold_back && issued == 0;
            const bool take = attn_take(p, cur.wanted, cur.block) && !held;
            const int n = __popc(__ballot_sync(0xffffffffu, take));
            if (lane == 0 && !held) mbar_arrive_expect_tx(full + 8 * stage, (uint32_t)(n * p.box * (2 * D + 2)));
            __syncwarp();
            if (take) {
                const uint32_t dst = base + stage * S::kStage + lane * p.box * D;
                copy_box(dst, &kmap, cur.token, cur.head, cur.block, full + 8 * stage);
                copy_box(dst + S::kHalf, &vmap, cur.token, cur.head, cur.block, full + 8 * stage);
                const int64_t byte = ((int64_t)cur.block * p.kv_heads + cur.head) * p.block_size + cur.token;
                const uint32_t to = base + S::kOffScale + stage * 2 * kAttnTile + lane * p.box;
                copy_bytes(to, p.scales[0] + byte, p.box, full + 8 * stage);
                copy_bytes(to + kAttnTile, p.scales[1] + byte, p.box, full + 8 * stage);
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
    float* row_scale = reinterpret_cast<float*>(sm + S::kOffRow);
    // [two][row][D], groups of 16 columns swizzled by the row
    float* merge = reinterpret_cast<float*>(sm + S::kOffMerge);
    for (; walk.next(); walk.done()) {
        const int q_off = S::kOffQ + (items & 1u) * S::kQ;
        wait(q_full + 8 * (items & 1u), (items >> 1) & 1u);
        // The queries in place into fp16 times a power of two that brings the
        // row's largest into [2^14, 2^15), four rows a warp. Of 16 dimensions
        // 4i, 4i+1 go to places 2i, 2i+1 and 4i+2, 4i+3 to 8+2i, 9+2i.
#pragma unroll
        for (int r = 0; r < kRows / kConsumers; ++r) {
            const int row = warp * (kRows / kConsumers) + r;
            if (row >= walk.rows) break;
            constexpr int kWords = D / 64;  // of two dimensions a lane
            uint32_t* words = reinterpret_cast<uint32_t*>(sm + q_off + row * S::kQRow);
            float2 v[kWords];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t w = words[lane * kWords + i];
                v[i] = DT == 0 ? make_float2(bf16lo(w), bf16hi(w)) : f16x2_to_f32(w);
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
            if (lane == 0) row_scale[row] = exp2i(-s) * p.scale_log2;
        }
        warps_sync(1, kConsumers * 32);
        // (rows past the item's last hold anything; a row's results depend on
        // no other row)
        const uint32_t q_addr = base + q_off + (lane & 15) * S::kQRow + (lane >> 4) * 16;
        const AllKeys all = attn_all_keys(walk, 0, walk.rows);
        const Tree tree = attn_tree<TREE>(walk);
        // of this thread's four rows (8 h + quad): the last key that each sees
        // and the first
        int last[4], from[4];
        float factor[4];
        unsigned long long mask[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const RowKeys k = attn_row_keys(walk, h * 8 + quad);
            last[h] = k.last;
            from[h] = k.from;
            factor[h] = row_scale[h * 8 + quad];
            mask[h] = TREE ? attn_tree_mask(walk, tree, h * 8 + quad) : ~0ull;
        }
        float o[2][D / 8][4];
        float m[4], w[4], l[4];  // references of the scores and of the products' weights
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            m[h] = w[h] = -INFINITY;
            l[h] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][i][j] = 0.f;
        const bool two = walk.rows > 16;  // sets of 16 rows
        for (int t = walk.t0; t < walk.t1; ++t) {
            if (!wait(full + 8 * stage, parity)) break;
            const int key0 = (walk.tile0 + t) * kAttnTile + warp * kWarpKeys;
            const uint32_t ks = base + stage * S::kStage, vs = ks + S::kHalf;
            if (attn_needs(walk, key0, kWarpKeys)) {
                const bool ragged = attn_ragged(walk, key0, kWarpKeys);
                // the exponents of this thread's four keys, 8 i + 2 pair + j
                float kf[4], ve[4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t* bytes = sm + S::kOffScale + stage * 2 * kAttnTile + warp * kWarpKeys + i * 8 + 2 * pair;
                    const uint32_t kb = *reinterpret_cast<const uint16_t*>(bytes), vb = *reinterpret_cast<const uint16_t*>(bytes + kAttnTile);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t a = (kb >> (8 * j)) & 255u, b = (vb >> (8 * j)) & 255u;
                        kf[2 * i + j] = e8m0_to_f32(a);
                        ve[2 * i + j] = b == 255u ? __uint_as_float(0x7fc00000u) : (float)((int)b - 127);
                    }
                }
                if (ragged) {
                    // values that no row sees may be anything: a weight of 0 times
                    // NaN is not 0, so they are cleared, and their exponents
                    const int key = key0 + (lane & 15);
                    if (key < walk.lo || key >= walk.hi) {
                        uint8_t* v = sm + stage * S::kStage + S::kHalf + (warp * kWarpKeys + (lane & 15)) * D + (lane >> 4) * (D / 2);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = key0 + (i >> 1) * 8 + 2 * pair + (i & 1);
                        if (k < walk.lo || k >= walk.hi) ve[i] = 0.f;
                    }
                    __syncwarp();
                }
                float s[2][2][4];
#pragma unroll
                for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[t2][i][j] = 0.f;
                const int k_row = warp * kWarpKeys + (lane & 7) + ((lane >> 4) << 3), k_piece = (lane >> 3) & 1;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t codes[4];
                    ldsm_x4(ks + piece_at<D>(k_row, 2 * c + k_piece), codes);
                    // codes of keys 0-7: dimensions 32 c .., 32 c + 16 ..; then
                    // of keys 8-15
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t b[2][2];
                        e4m3x4_to_f16x2(codes[k], b[0][0], b[0][1]);
                        e4m3x4_to_f16x2(codes[2 + k], b[1][0], b[1][1]);
                        uint32_t a[4];
                        ldsm_x4(q_addr + (2 * c + k) * 32, a);
                        mma_f16(s[0][0], a, b[0][0], b[0][1]);
                        mma_f16(s[0][1], a, b[1][0], b[1][1]);
                        if (two) {
                            ldsm_x4(q_addr + 16 * S::kQRow + (2 * c + k) * 32, a);
                            mma_f16(s[1][0], a, b[0][0], b[0][1]);
                            mma_f16(s[1][1], a, b[1][0], b[1][1]);
                        }
                    }
                }
                // scores in units of log2, element (i, j & 1) of row half j >> 1
                const bool some = all.lacks(key0, kWarpKeys), leaves = TREE && tree.reaches(key0, kWarpKeys);
                bool grows = false;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h >= 2 && !two) break;
                    float big = -INFINITY, big_v = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float& x = s[h >> 1][e >> 1][(h & 1) * 2 + (e & 1)];
                        x *= factor[h] * kf[e];
                        if (some || leaves) {
                            const int key = key0 + (e >> 1) * 8 + 2 * pair + (e & 1);
                            if (key > last[h] || key < from[h]) x = -INFINITY;
                            if (TREE && attn_tree_hides(tree, mask[h], key)) x = -INFINITY;
                        }
                        big = fmaxf(big, x);
                        big_v = fmaxf(big_v, x + ve[e]);
                    }
                    grows |= big > m[h] + kLimit || big_v > w[h] + kLimit;
                }
                // (rare: the largest scores so far move up by more than 2^4 a
                // few times in a row of any length)
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        if (h >= 2 && !two) break;
                        float big = -INFINITY, big_v = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = s[h >> 1][e >> 1][(h & 1) * 2 + (e & 1)];
                            big = fmaxf(big, x);
                            big_v = fmaxf(big_v, x + ve[e]);
                        }
#pragma unroll
                        for (int d = 1; d < 4; d <<= 1) {
                            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
                            big_v = fmaxf(big_v, __shfl_xor_sync(0xffffffffu, big_v, d));
                        }
                        if (big > m[h] + kLimit) {
                            l[h] *= exp2_approx(m[h] - (big - kBias));
                            m[h] = big - kBias;
                        }
                        const bool up = big_v > w[h] + kLimit;
                        const float f = up ? exp2_approx(w[h] - (big_v - kBias)) : 1.f;
                        if (up) w[h] = big_v - kBias;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[h >> 1][i][(h & 1) * 2] *= f;
                            o[h >> 1][i][(h & 1) * 2 + 1] *= f;
                        }
                    }
                }
                uint32_t pa[2][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h >= 2 && !two) break;
                    const float ref = m[h] == -INFINITY ? 0.f : m[h], ref_v = w[h] == -INFINITY ? 0.f : w[h];
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = s[h >> 1][i][(h & 1) * 2], y = s[h >> 1][i][(h & 1) * 2 + 1];
                        sum += exp2_approx(x - ref) + exp2_approx(y - ref);
                        pa[h >> 1][i * 2 + (h & 1)] =
                            f32x2_to_f16x2(exp2_approx(x + (ve[2 * i] - ref_v)), exp2_approx(y + (ve[2 * i + 1] - ref_v)));
                    }
                    l[h] += sum;
                }
                const int v_row = warp * kWarpKeys + (lane & 15), v_piece = lane >> 4;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t codes[4];
                    ldsm_x4_trans(vs + piece_at<D>(v_row, 2 * c + v_piece), codes);
                    // two keys' codes of dimensions 2i and 2i + 1: of 16
                    // dimensions keys 0-7 and 8-15, then of the next 16
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        uint32_t even[2], odd[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) e4m3x4_to_f16x2(__byte_perm(codes[2 * g + k], 0, 0x3120), even[k], odd[k]);
                        mma_f16(o[0][4 * c + 2 * g], pa[0], even[0], even[1]);
                        mma_f16(o[0][4 * c + 2 * g + 1], pa[0], odd[0], odd[1]);
                        if (two) {
                            mma_f16(o[1][4 * c + 2 * g], pa[1], even[0], even[1]);
                            mma_f16(o[1][4 * c + 2 * g + 1], pa[1], odd[0], odd[1]);
                        }
                    }
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
        // (this warp's rows of the queries were written in place: the next copy
        // into them comes after)
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty + 8 * (items & 1u));
        ++items;
        // join the warps: each scales to the largest score of all, then they add
        // up one after another, four in each of two places
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            if (pair == 0) stat[warp * kRows + h * 8 + quad] = make_float2(m[h], l[h]);
        }
        warps_sync(1, kConsumers * 32);
        float all_m[4], all_l[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int row = h * 8 + quad;
            float mx = -INFINITY, tot = 0.f;
#pragma unroll
            for (int x = 0; x < kConsumers; ++x) mx = fmaxf(mx, stat[x * kRows + row].x);
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int x = 0; x < kConsumers; ++x) tot += stat[x * kRows + row].y * exp2_approx(stat[x * kRows + row].x - ref);
            all_m[h] = mx;
            all_l[h] = tot;
            const float f = exp2_approx(w[h] - ref);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[h >> 1][i][(h & 1) * 2] *= f;
                o[h >> 1][i][(h & 1) * 2 + 1] *= f;
            }
        }
        for (int x = 0; x < kConsumers / 2; ++x) {
            if (warp / 2 == x) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (h >= 2 && !two) break;
                    // dimensions 16 g + 4 pair .. + 3
                    float* row = merge + (warp & 1) * (kRows * D) + (h * 8 + quad) * D + 4 * pair;
#pragma unroll
                    for (int g = 0; g < D / 16; ++g) {
                        float4* to = reinterpret_cast<float4*>(row + (g ^ (quad & 1)) * 16);
                        float4 u = x > 0 ? *to : make_float4(0.f, 0.f, 0.f, 0.f);
                        u.x += o[h >> 1][2 * g][(h & 1) * 2];
                        u.y += o[h >> 1][2 * g + 1][(h & 1) * 2];
                        u.z += o[h >> 1][2 * g][(h & 1) * 2 + 1];
                        u.w += o[h >> 1][2 * g + 1][(h & 1) * 2 + 1];
                        *to = u;
                    }
                }
            }
            // (everyone has read the statistics by the first of these)
            if (x == kConsumers / 2 - 1 && warp == 0 && pair == 0)
#pragma unroll
                for (int h = 0; h < 4; ++h) stat[h * 8 + quad] = make_float2(all_m[h], all_l[h]);
            warps_sync(1, kConsumers * 32);
        }
        // 16 bytes of output a thread
        const bool whole = walk.whole();
        float* part = p.part + ((int64_t)blockIdx.x * 2 + walk.part()) * attn_part_floats(kRows, D);
        for (int i = tid; i < walk.rows * (D / 8); i += kConsumers * 32) {
            const int row = i / (D / 8), c = i % (D / 8);
            const float* from_row = merge + row * D + ((c >> 1) ^ (row & 1)) * 16 + (c & 1) * 8;
            float4 x = *reinterpret_cast<const float4*>(from_row), y = *reinterpret_cast<const float4*>(from_row + 4);
            const float4 x2 = *reinterpret_cast<const float4*>(from_row + kRows * D), y2 = *reinterpret_cast<const float4*>(from_row + kRows * D + 4);
            x.x += x2.x; x.y += x2.y; x.z += x2.z; x.w += x2.w;
            y.x += y2.x; y.y += y2.y; y.z += y2.z; y.w += y2.w;
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
