// What the kernels of attention over the paged cache share: the place of a
// CTA in the work, the joining of parts, bounded waits, tensor-map copies of
// pages.
#pragma once
#include <cuda.h>

#include "attn_work.cuh"
#include "ptx.cuh"

namespace moe {

constexpr float kLn2 = 0.693147180559945f;

// Finds the CTA's range and the item that it begins in, all threads together:
// one of them walks to the item, for all. `scan` is shared memory of THREADS /
// 32 values.
template <class Class, int THREADS>
__device__ __forceinline__ Place attn_place(const AttnParams& p, int cta, int64_t* scan, Start* found) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int r0 = min(tid * per, p.B), r1 = min(r0 + per, p.B);
    int64_t own = 0;
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const Request q = attn_request(p, r);
        bad |= q.bad;
        if (Class::mine(p, q)) own += attn_request_units<Class>(p, q) * p.kv_heads;
    }
    if (bad) atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
    int64_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    Place at;
    at.total = 0;
    int64_t before = sum - own;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += scan[w];
        at.total += scan[w];
    }
    attn_range(p, cta, at);
    if (own > 0 && before <= at.begin && at.begin < before + own) *found = attn_seek<Class>(p, r0, r1, at.begin - before);
    __syncthreads();
    at.start = *found;  // (anything, for a CTA without units)
    return at;
}

// A barrier of some of the CTA's warps. (bar.sync is .aligned: it asks for whole
// warps, and what comes before is often some lanes'.)
__device__ __forceinline__ void warps_sync(uint32_t id, uint32_t threads) {
    __syncwarp();
    named_bar_sync(id, threads);
}

// One thread of a CTA whose part is in place (its threads' stores are behind a
// barrier): whether all the others are. The last one to come leaves the count
// at zero for the next call.
__device__ __forceinline__ bool attn_last(unsigned* arrived, int parts) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(arrived) : "memory");
    if (old != (unsigned)parts - 1) return false;
    asm volatile("st.relaxed.gpu.global.u32 [%0], 0;" ::"l"(arrived) : "memory");
    return true;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
__device__ __forceinline__ float exp2_approx(float x);

// (A sum of weights is 0, NaN or above 0: NaN has to reach the output and lse.)
// Joins the parts of an item, in the order of the keys (the part 1 of the CTA
// that it begins in, then the part 0 of the CTAs after it): THREADS threads,
// the rows [from, to). A thread takes U pieces of 8 dimensions at a time, all
// their loads of a part in flight together.
template <int D, int DT, int ROWS, int THREADS, int U>
__device__ __forceinline__ void attn_join(const AttnParams& p, const float* parts, const Span& span, int from, int to,
                                          int row0, int head, int token0, int tid) {
    constexpr int kFloats = attn_part_floats(ROWS, D), kPer = D / 8;
    const float* first = parts + ((int64_t)span.cta * 2 + 1) * kFloats;
    const float* rest = parts + (int64_t)span.cta * 2 * kFloats;  // part 0 of the k-th CTA at k * 2 * kFloats
    auto part_of = [&](int k) { return k == 0 ? first : rest + (int64_t)k * 2 * kFloats; };
    auto stat_of = [&](int k, int row) { return __ldcg(reinterpret_cast<const float2*>(part_of(k) + ROWS * D) + row); };
    const int end = to * kPer;
    for (int i0 = tid + from * kPer; i0 < end; i0 += U * THREADS) {
        // (past the end the last piece again, not stored)
        float mx[U], sum[U], v[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            mx[u] = -INFINITY;
            sum[u] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 0.f;
        }
#pragma unroll 2
        for (int k = 0; k < span.parts; ++k)
#pragma unroll
            for (int u = 0; u < U; ++u) mx[u] = fmaxf(mx[u], stat_of(k, min(i0 + u * THREADS, end - 1) / kPer).x);
        for (int k = 0; k < span.parts; ++k) {
            float2 ml[U];
            float4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = min(i0 + u * THREADS, end - 1);
                const float4* f = reinterpret_cast<const float4*>(part_of(k) + (int64_t)i * 8);
                ml[u] = stat_of(k, i / kPer);
                x[u] = __ldcg(f);
                y[u] = __ldcg(f + 1);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = exp2_approx(ml[u].x - (mx[u] == -INFINITY ? 0.f : mx[u]));
                sum[u] += w * ml[u].y;
                v[u][0] += w * x[u].x; v[u][1] += w * x[u].y; v[u][2] += w * x[u].z; v[u][3] += w * x[u].w;
                v[u][4] += w * y[u].x; v[u][5] += w * y[u].y; v[u][6] += w * y[u].z; v[u][7] += w * y[u].w;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * THREADS;
            if (i >= end) break;
            const int row = i / kPer, d = (i % kPer) * 8;
            const float inv = sum[u] != 0.f ? 1.f / sum[u] : 0.f;
            const int R = row0 + row, t = token_of(p, R), h = head * p.group + (R - t * p.group);
            const int64_t at_row = (int64_t)(token0 + t) * p.heads + h;
            uint4 o;
            o.x = pack2<DT>(v[u][0] * inv, v[u][1] * inv);
            o.y = pack2<DT>(v[u][2] * inv, v[u][3] * inv);
            o.z = pack2<DT>(v[u][4] * inv, v[u][5] * inv);
            o.w = pack2<DT>(v[u][6] * inv, v[u][7] * inv);
            *reinterpret_cast<uint4*>(p.out + at_row * D + d) = o;
            if (d == 0 && p.lse) p.lse[at_row] = sum[u] != 0.f ? (mx[u] + log2f(sum[u])) * kLn2 : -INFINITY;
        }
    }
}

// A part of the chunk kernel: for each slot of 128 rows four dimensions of all
// rows after another, so that a warp's 32 rows are stored and read together;
// then the rows' largest scores and sums. The join, a thread a row: bound by
// what one SM reads from the L2 (two slots of 128 dimensions in five parts,
// 640 KB, take 14,000 cycles; 33,000 with rows of the part side by side).
template <int D, int DT>
__device__ __noinline__ void attn_join_slot(const AttnParams& p, const float* parts, const Span& span, int slot, int row,
                                               int64_t at_row, bool real) {
    constexpr int kFloats = attn_part_floats(kAttnChunkRows, D), kSlot = 128;
    const float* first = parts + ((int64_t)span.cta * 2 + 1) * kFloats;
    const float* rest = parts + (int64_t)span.cta * 2 * kFloats;  // part 0 of the k-th CTA at k * 2 * kFloats
    auto part_of = [&](int k) { return k == 0 ? first : rest + (int64_t)k * 2 * kFloats; };
    auto stat_of = [&](int k) {
        return __ldcg(reinterpret_cast<const float2*>(part_of(k) + kAttnChunkRows * D) + slot * kSlot + row);
    };
    float mx = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int k = 0; k < span.parts; ++k) mx = fmaxf(mx, stat_of(k).x);
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int k = 0; k < span.parts; ++k) {
        const float2 ml = stat_of(k);
        sum += exp2_approx(ml.x - ref) * ml.y;
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    constexpr int kStep = 16;  // 16-byte loads in flight
#pragma unroll
    for (int c0 = 0; c0 < D / 4; c0 += kStep) {
        float4 v[kStep];
#pragma unroll
        for (int c = 0; c < kStep; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < span.parts; ++k) {
            const float4* f = reinterpret_cast<const float4*>(part_of(k)) + (slot * (D / 4) + c0) * kSlot + row;
            float4 x[kStep];
#pragma unroll
            for (int c = 0; c < kStep; ++c) x[c] = __ldcg(f + c * kSlot);
            const float w = exp2_approx(stat_of(k).x - ref) * inv;
#pragma unroll
            for (int c = 0; c < kStep; ++c) {
                v[c].x += w * x[c].x;
                v[c].y += w * x[c].y;
                v[c].z += w * x[c].z;
                v[c].w += w * x[c].w;
            }
        }
        if (!real) continue;
#pragma unroll
        for (int c = 0; c < kStep; c += 2) {
            uint4 o;
            o.x = pack2<DT>(v[c].x, v[c].y);
            o.y = pack2<DT>(v[c].z, v[c].w);
            o.z = pack2<DT>(v[c + 1].x, v[c + 1].y);
            o.w = pack2<DT>(v[c + 1].z, v[c + 1].w);
            *reinterpret_cast<uint4*>(p.out + at_row * D + (c0 + c) * 4) = o;
        }
    }
    if (real && p.lse) p.lse[at_row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

// Waits for the phase with parity `parity`, at most timeout_ns; false, with
// the status and `flag` set, when it ran out or another wait of the CTA did.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, const AttnParams& p, volatile int* flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*flag) return false;
        if (global_timer_ns() - t0 > p.timeout_ns) {
            atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -101 /* MOE_ETIMEOUT */);
            *flag = 1;
            return false;
        }
    }
    return true;
}

// Waits for the phase with parity `parity` of work that the CTA itself has
// issued: copies into its shared memory, products in its tensor memory. Both
// belong to the next CTA once this one has ended, so whoever issued something
// sees it done before it leaves, whether a wait of the CTA has run out or not,
// and with a limit of its own: the option's may be short.
constexpr uint64_t kDrainNs = 2000000000;
__device__ __forceinline__ void attn_drain(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kDrainNs) {
    }
}

// One box of a cache's tensor map (64 dimensions, token of the block, which 64,
// head, block) into shared memory: `box` keys, 128 bytes a key in the 128-byte
// swizzle, one panel of 64 dimensions after another. The innermost coordinate
// is always 0.
__device__ __forceinline__ void attn_copy(uint32_t dst, const CUtensorMap* map, int panel, int token, int head,
                                          int block, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(map), "r"(0), "r"(token), "r"(panel), "r"(head), "r"(block), "r"(bar)
        : "memory");
}

// Whether the box is copied: wanted and in a block that there is.
__device__ __forceinline__ bool attn_take(const AttnParams& p, bool wanted, int block) {
    if (wanted && (unsigned)block >= (unsigned)p.n_blocks) {
        atomicCAS(reinterpret_cast<int*>(p.ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
        return false;
    }
    return wanted;
}

// The softmax weights are 2^(score - m). The reference m of a row is set kBias
// below its largest score and stays until a score is more than kLimit above it,
// so most tiles need no pass over the sums. bf16 has fp32's exponents. fp16 ends
// at 2^-24: next to a largest weight of 1 many keys of 2^-25 each would be lost
// (60,000 of them are 0.2% of the output), so its weights reach up to 2^15 and
// the least that it holds is 2^-35 of the largest.
template <int DT>
struct WeightRange {
    static constexpr float kBias = DT == 0 ? 0.f : 11.f, kLimit = DT == 0 ? 8.f : 15.f;
};

// Two fp32 into one register of the type, `lo` in the low half (one rounding).
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t d;
    if (DT == 0) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace moe
