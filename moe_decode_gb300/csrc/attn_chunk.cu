// Attention of many query rows over the paged cache (prompt chunks, long verify
// blocks times their grouped heads) on the 5th-generation tensor cores.
//
// One pass over the keys with a running reference m and sum l per row: S = Q
// K^T, P = 2^(c S - m), l += sum P, O += P V, O / l at the end. An item is two
// tiles of 128 query rows (slots) against the same keys. For each tile of 128
// keys and each slot, one thread issues S = Q K^T (both from shared memory in
// the 128-byte swizzle) into tensor memory; the slot's four warps, one thread
// a row, turn S into P and write it over S in 16 bits; O += P V takes P from
// tensor memory and V from shared memory as it lies (keys by dimensions, the
// dimensions contiguous). While one slot's warps work on their tile the tensor
// core works for the other slot: the order is PV(slot, j), QK(slot, j + 1) for
// slot 0, then for slot 1, and each completion that lets a slot's warps read
// S(j + 1) also says that PV(j) is done, so they may rescale O. They do so only
// where the largest score of a row has left the reference's range.
//
// Two chunks of 8,192 tokens over 16,383 keys (32/8 heads of 128) take 2.58 ms
// replayed from a graph, 1,280 TFLOP/s (2.09 ms with heads of 64). A tile of both slots takes 3,500 cycles where its products
// alone are 2,048: 1,580 of a slot's softmax, 1,024 of its products and 500 to
// 900 of hand-overs and of waiting for shared memory, which brings the 128
// bytes a clock that Q K^T with both operands from it wants (without any
// softmax the call takes 2.17 ms).
#include "attn_common.cuh"

namespace moe {
namespace {

constexpr int kSlotRows = 128;
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kThreads = 384;  // two warpgroups of softmax, one for the two issuing warps
// A thread of the softmax holds a row of 128 scores: its warpgroups take
// registers from the third. Together exactly what the block is launched with.
// (At 128 dimensions 360 bytes of stores and 504 of loads are spilled.)
constexpr int kLaunchRegs = 168, kSoftmaxRegs = 216, kIssueRegs = 72;
static_assert(2 * kSoftmaxRegs + kIssueRegs == 3 * kLaunchRegs, "registers of the block");

template <int D>
struct ChunkShape {
    static constexpr int kPanel = 128 * 128;            // 128 rows of 64 dimensions
    static constexpr int kTile = kPanel * (D / 64);     // Q of a slot, K or V of a tile
    static constexpr int kStages = D == 128 ? 5 : 10;   // K and V in turn
    static constexpr int kOffKv = 2 * kTile;
    static constexpr int kOffBar = kOffKv + kStages * kTile;
    static constexpr int kBytes = kOffBar + 512 + 1024;  // and room to align
    static constexpr uint32_t kColO = 256;               // tensor memory: S0, S1, then O0, O1
};

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// d (+)= a b, both from shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// d (+)= a b, a from tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// 32 columns of this warp's 32 lanes, one lane a thread.
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand in the 128-byte swizzle: rows of 128 bytes, groups of
// eight rows 1,024 bytes apart. `lead` is the distance of the 64-element
// panels where the operand's contiguous dimension is not the summed one.
// The low word of the descriptor (address, lead); the high word is the same
// for all.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lead) {
    return ((addr & 0x3ffffu) >> 4) | ((lead >> 4) << 16);
}
__device__ __forceinline__ uint64_t descriptor(uint32_t low) {
    constexpr uint32_t high = (1024 >> 4) | (1u << 14) | (2u << 29);
    return ((uint64_t)high << 32) | low;
}
// fp32 sums, 16-bit operands of the type, 128 rows, n columns; `across`: the
// second operand's contiguous dimension is its column.
template <int DT>
__device__ constexpr uint32_t product(uint32_t n, bool across) {
    return (1u << 4) | ((DT == 0 ? 1u : 0u) << 7) | ((DT == 0 ? 1u : 0u) << 10) | ((across ? 1u : 0u) << 16) |
           ((n >> 3) << 17) | ((128u >> 4) << 24);
}

template <int D, int DT>
__global__ __launch_bounds__(kThreads, 1) void attn_chunk_kernel(const __grid_constant__ AttnParams p,
                                                                  const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap) {
    using S = ChunkShape<D>;
    extern __shared__ uint8_t dyn[];
    __shared__ int64_t scan[kThreads / 32];
    __shared__ Start found;
    __shared__ int abort_flag;
    __shared__ int join_info[2][3];  // first CTA, parts, whether this one is the last
    __shared__ uint32_t tmem_base;
    const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
    uint8_t* sm = dyn + (base - smem_u32(dyn));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // barriers: key/value stages full and empty; per slot queries in place, S
    // written, P written, O complete; the last products of the CTA
    const uint32_t full = base + S::kOffBar, empty = full + 8 * S::kStages;
    const uint32_t q_full = empty + 8 * S::kStages, s_full = q_full + 16, p_full = s_full + 16, o_full = p_full + 16,
                   drained = o_full + 16;
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(q_full + 8 * t, kSlotRows);
            mbar_init(s_full + 8 * t, 1 + p.hold_back);  // (held back: a second arrival that never comes)
            mbar_init(p_full + 8 * t, kSlotRows);
            mbar_init(o_full + 8 * t, 1);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    // The decode kernel runs before this one, and lets it start once its own
    // wait for what came before is over; none of its results are needed here,
    // so the two overlap (all reads go to the L2, where what came before is).
    // The wait at the end keeps the order for what follows.
    pdl_launch_dependents();
    const Place at = attn_place<Many, kThreads>(p, blockIdx.x, scan, &found);
    if (at.begin >= at.end) {
        pdl_wait();
        return;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_base))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    volatile int* flag = &abort_flag;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == kLoadWarp) {
            // lane i brings the tile's i-th box, if a row sees any of it; K of a
            // tile, then V
            int stage = 0, issued = 0;
            uint32_t parity = 1;
            bool ok = true;
            TileFeed<Many> feed(p, at, lane);
            auto cur = feed.box(), next = cur;
            for (bool more = feed.any; ok && more; cur = next) {
                more = feed.advance();
                if (more) next = feed.box();
                const bool take = attn_take(p, cur.wanted, cur.block);
                const int n = __popc(__ballot_sync(0xffffffffu, take));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xffffffffu, ok && attn_wait(empty + 8 * stage, parity, p, flag));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(full + 8 * stage, (uint32_t)(n * p.box * D * 2));
                    __syncwarp();
                    if (take) {
                        const uint32_t dst = base + S::kOffKv + stage * S::kTile + lane * p.box * 128;
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            attn_copy(dst + x * S::kPanel, kv ? &vmap : &kmap, x, cur.token, cur.head, cur.block,
                                      full + 8 * stage);
                    }
                    ++issued;
                    if (++stage == S::kStages) {
                        stage = 0;
                        parity ^= 1u;
                    }
                }
            }
            // the last copies of each stage, in flight where another role gave up
            if (lane == 0)
                for (int i = max(0, issued - S::kStages); i < issued; ++i)
                    attn_drain(full + 8 * (i % S::kStages), (uint32_t)((i / S::kStages) & 1));
            __syncwarp();
        } else if (warp == kMmaWarp) {
            if (lane == 0) {
                Walk<Many> walk(p, at);
                uint32_t pos = 0;  // stages consumed
                uint32_t q_par = 0, p_par = 0;  // parity bits by slot
                bool ok = true;
                auto arrived = [&](uint32_t i) { return attn_wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1u, p, flag); };
                auto scores = [&](int t, uint32_t i) {
                    const uint32_t a = operand(base + t * S::kTile, 16);
                    const uint32_t b = operand(base + S::kOffKv + (i % S::kStages) * S::kTile, 16);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k >> 2) * S::kPanel + (k & 3) * 32) >> 4;
                        tc_mma_ss(tmem + t * 128, descriptor(a + off), descriptor(b + off), product<DT>(128, false), k > 0);
                    }
                    tc_commit(s_full + 8 * t);
                };
                for (; ok && walk.next(); walk.done()) {
                    const int slots = walk.rows > kSlotRows ? 2 : 1, n = walk.t1 - walk.t0;
                    for (int t = 0; ok && t < slots; ++t) {
                        ok = attn_wait(q_full + 8 * t, (q_par >> t) & 1u, p, flag);
                        q_par ^= 1u << t;
                    }
                    ok = ok && arrived(pos);
                    if (!ok) break;
                    tc_fence_after();
                    for (int t = 0; t < slots; ++t) scores(t, pos);
                    tc_commit(empty + 8 * (pos % S::kStages));
                    ++pos;
                    for (int j = 0; ok && j < n; ++j) {
                        const bool more = j + 1 < n;
                        ok = arrived(pos) && (!more || arrived(pos + 1));
                        for (int t = 0; ok && t < slots; ++t) {
                            ok = attn_wait(p_full + 8 * t, (p_par >> t) & 1u, p, flag);
                            if (!ok) break;
                            p_par ^= 1u << t;
                            tc_fence_after();
                            const uint32_t b = operand(base + S::kOffKv + (pos % S::kStages) * S::kTile, S::kPanel);
#pragma unroll
                            for (int k = 0; k < kAttnTile / 16; ++k)
                                tc_mma_ts(tmem + S::kColO + t * D, tmem + t * 128 + k * 8, descriptor(b + k * (2048 >> 4)),
                                          product<DT>(D, true), j > 0 || k > 0);
                            if (more) scores(t, pos + 1);
                            else tc_commit(o_full + 8 * t);
                        }
                        if (!ok) break;
                        tc_commit(empty + 8 * (pos % S::kStages));
                        if (more) tc_commit(empty + 8 * ((pos + 1) % S::kStages));
                        pos += more ? 2 : 1;
                    }
                }
                // the last products, in flight where another role gave up: tensor
                // memory is freed after them
                tc_commit(drained);
                attn_drain(drained, 0);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        Walk<Many> walk(p, at);
        const int slot = warp >> 2, t = tid & (kSlotRows - 1);
        const int row = t;  // of the slot: that of the warp's lanes of tensor memory
        auto piece_at = [&](int slot, int row, int c) {  // 16 bytes of a slot's row
            return slot * S::kTile + (c >> 3) * S::kPanel + row * 128 + (((c & 7) ^ (row & 7)) << 4);
        };
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t s_at = lanes + slot * 128, o_at = lanes + S::kColO + slot * D;
        uint32_t s_par = 0, o_par = 0;
        uint32_t pos = 0;  // stages of the items before
        // A wait that ran out ends the work of the warp, but not its way past the
        // barriers that others of its slot stand at.
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && attn_wait(bar, parity, p, flag));
            return ok;
        };
        for (; walk.next(); walk.done()) {
            const int n = walk.t1 - walk.t0;
            const uint32_t first_stage = pos;
            pos += 2 * n;
            if (slot * kSlotRows >= walk.rows) continue;
            const int slot_row0 = walk.row0 + slot * kSlotRows;
            const int slot_rows = min(kSlotRows, walk.rows - slot * kSlotRows);
            const int R = slot_row0 + row;
            const bool real = row < slot_rows;
            const int tok = token_of(p, R), head = walk.head * p.group + (R - tok * p.group);
            // the slot's rows into shared memory, 16-byte pieces in the swizzle
            // (a row's pieces by neighbouring threads); rows past the end are
            // zeros
            {
                constexpr int kPer = D / 8;
                uint4 v[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    // (the last row again for those past the end: all the loads
                    // are on their way before the first is waited for)
                    const int g = i * kSlotRows + t, at_R = slot_row0 + min(g / kPer, slot_rows - 1);
                    const int q_tok = token_of(p, at_R), q_head = walk.head * p.group + (at_R - q_tok * p.group);
                    v[i] = __ldcg(reinterpret_cast<const uint4*>(p.q + (walk.q.q0 + q_tok) * p.q_token +
                                                                 q_head * p.q_head + (g % kPer) * 8));
                }
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int g = i * kSlotRows + t;
                    *reinterpret_cast<uint4*>(sm + piece_at(slot, g / kPer, g % kPer)) =
                        g / kPer < slot_rows ? v[i] : make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
                mbar_arrive(q_full + 8 * slot);
            }
            // keys that the row sees, and that all or any rows of the slot see
            const RowKeys sees = attn_row_keys(walk, slot * kSlotRows + row);
            const AllKeys all = attn_all_keys(walk, slot * kSlotRows, slot * kSlotRows + slot_rows);
            float m = -INFINITY;  // reference of the weights, in log2
            float l = 0.f;
            for (int j = 0; j < n; ++j) {
                const int key0 = (walk.tile0 + walk.t0 + j) * kAttnTile;
                if (!wait(s_full + 8 * slot, s_par)) break;
                s_par ^= 1u;
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(s_at + 32 * c, s + 32 * c);
                tc_wait_ld();
                if (all.lacks(key0, kAttnTile)) {
#pragma unroll
                    for (int i = 0; i < 128; ++i)
                        if (key0 + i > sees.last || key0 + i < sees.from) s[i] = 0xff800000u;  // -inf
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 128; i += 4)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(s[i + k]));
                const float big = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                const bool grows = big > m + WeightRange<DT>::kLimit;
                const float to = big - WeightRange<DT>::kBias;
                if (__any_sync(0xffffffffu, grows)) {
                    const float f = grows ? exp2_approx(m - to) : 1.f;
                    if (grows) m = to;
                    l *= f;
                    if (j > 0) {
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tc_ld32(o_at + 32 * c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc_st32(o_at + 32 * c, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), ref2 = make_float2(-ref, -ref);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int k = 64 * h + 2 * i;
                        float2 x = ffma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), scale2, ref2);
                        x.x = exp2_approx(x.x);
                        x.y = exp2_approx(x.y);
                        sum[i & 1] = __fadd2_rn(sum[i & 1], x);
                        // rounded once to the values' type for the second
                        // product; the sum keeps the fp32 weights
                        s[32 * h + i] = pack2<DT>(x.x, x.y);
                    }
                    tc_st32(s_at + 32 * h, s + 32 * h);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                // values that no row sees may be anything: a weight of 0 times
                // NaN is not 0, so they are cleared
                if (slot == 0 && attn_ragged(walk, key0, kAttnTile)) {
                    const uint32_t i = first_stage + 2 * j + 1;
                    if (!wait(full + 8 * (i % S::kStages), (i / S::kStages) & 1u)) break;
                    if (key0 + row < walk.lo || key0 + row >= walk.hi) {
                        uint8_t* v = sm + S::kOffKv + (i % S::kStages) * S::kTile + row * 128;
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(v + x * S::kPanel + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_shared();
                }
                __syncwarp();  // (some rows' threads cleared values)
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(p_full + 8 * slot);
            }
            wait(o_full + 8 * slot, o_par);
            o_par ^= 1u;
            tc_fence_after();
            const bool whole = walk.whole();
            const float inv = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;
            const int64_t at_row = (int64_t)(walk.q.q0 + tok) * p.heads + head;
            float* part = p.chunk_part + ((int64_t)blockIdx.x * 2 + walk.part()) * attn_part_floats(kAttnChunkRows, D);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc_ld32(o_at + 32 * c, o);
                tc_wait_ld();
                if (whole) {
                    // by way of the queries' place, which is free
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint4 v;
                        v.x = pack2<DT>(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                        v.y = pack2<DT>(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
                        v.z = pack2<DT>(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv);
                        v.w = pack2<DT>(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv);
                        *reinterpret_cast<uint4*>(sm + piece_at(slot, row, 4 * c + i / 8)) = v;
                    }
                } else {
                    float4* to = reinterpret_cast<float4*>(part) + (slot * (D / 4) + 8 * c) * kSlotRows + row;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        to[i * kSlotRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                        __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                }
            }
            if (whole) {
                warps_sync(1 + slot, kSlotRows);
                constexpr int kPer = D / 8;
                // (each thread reads the pieces that it writes with the next
                // item's queries, so no barrier follows)
#pragma unroll 4
                for (int i = 0; i < kPer; ++i) {
                    const int g = i * kSlotRows + t, c = g % kPer, at_R = slot_row0 + g / kPer;
                    const uint4 v = *reinterpret_cast<const uint4*>(sm + piece_at(slot, g / kPer, c));
                    if (g / kPer < slot_rows) {
                        const int o_tok = token_of(p, at_R), o_head = walk.head * p.group + (at_R - o_tok * p.group);
                        *reinterpret_cast<uint4*>(p.out + ((int64_t)(walk.q.q0 + o_tok) * p.heads + o_head) * D + c * 8) = v;
                    }
                }
                if (real && p.lse) p.lse[at_row] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            } else {
                reinterpret_cast<float2*>(part + kAttnChunkRows * D)[slot * kSlotRows + row] = make_float2(m, l);
                warps_sync(1 + slot, kSlotRows);
                if (t == 0) {
                    const Span span = attn_span(walk, at);
                    join_info[slot][0] = span.cta;
                    join_info[slot][1] = span.parts;
                    join_info[slot][2] = attn_last(p.arrived + (1 + slot) * kAttnMaxGrid + span.cta, span.parts);
                }
                warps_sync(1 + slot, kSlotRows);
                if (join_info[slot][2])
                    attn_join_slot<D, DT>(p, p.chunk_part, Span{join_info[slot][0], join_info[slot][1]}, slot, row, at_row, real);
                warps_sync(1 + slot, kSlotRows);
            }
            // O is read: the next item's first product may write it
            tc_fence_before();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D, int DT>
cudaError_t launch_typed(const AttnParams& p, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    auto* kern = attn_chunk_kernel<D, DT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkShape<D>::kBytes);
    if (e != cudaSuccess) return e;
    // the warpgroups' shares wait for ever where the launch brings fewer
    cudaFuncAttributes have;
    e = cudaFuncGetAttributes(&have, kern);
    if (e != cudaSuccess) return e;
    if (have.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.G);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = ChunkShape<D>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, k, v);
}

}  // namespace

cudaError_t launch_attn_chunk(const AttnParams& p, const void* k_map, const void* v_map, int head_dim, int dtype,
                              cudaStream_t stream) {
    const CUtensorMap& k = *static_cast<const CUtensorMap*>(k_map);
    const CUtensorMap& v = *static_cast<const CUtensorMap*>(v_map);
    if (head_dim == 128) return dtype == 0 ? launch_typed<128, 0>(p, k, v, stream) : launch_typed<128, 1>(p, k, v, stream);
    return dtype == 0 ? launch_typed<64, 0>(p, k, v, stream) : launch_typed<64, 1>(p, k, v, stream);
}

}  // namespace moe
