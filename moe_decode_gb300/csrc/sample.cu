// Sampling from the output layer's logits with temperature, top-k, top-p and
// min-p, from given random numbers (moe_sample).
//
// Weights. t_i = (max - l_i) log2(e) / T in two fp32 parts (the difference and
// the product with their rounding errors), w_i = 2^-t_i as a 64-bit integer in
// units of 2^-42. Sums of integers do not depend on their order, so neither
// the split over CTAs nor atomics change a result, and a cumulated mass over
// 157,184 tokens keeps the relative error of its terms (one rounding of the
// fp32 mantissa), which a sum in fp32 would not: the token changes when a
// border of the cumulated mass moves across u * total.
//
// One cluster a row: each CTA keeps its slice of the row in shared memory, so
// the logits are read from HBM once. The kept set is a prefix of the order (l
// descending, index ascending), encoded in 55 bits as (t in 2^-17 steps, the
// bits of l reversed); top-k and top-p each look for its last member.
//
// Top-k. The largest logits of the threads, one each, are members too, so the
// bin in which k of them are reached cannot lie before the last member's: a
// histogram (512 bins of the code, summed across the cluster through
// distributed shared memory) that takes one atomic a thread, not one a logit.
// Nothing beyond its bin needs more than a subtraction, a product and a
// comparison from then on. Where at most kList members are left the first CTA
// ranks them, with top-p at once.
//
// Top-p otherwise. One sweep sums the masses and counts the members of each
// bin; their counts and mean places bound the masses to 10^-3, and so the
// border to a bin or two. A second sweep sums the masses before those exactly,
// with a histogram (count and mass) of those alone, in 512 parts.
//
// Either way the last member's bin is split again until it has at most kList
// members, which are ranked, or is one value, whose members count in index
// order.
#include <atomic>

#include "host.h"
#include "paged.h"
#include "ptx.cuh"

namespace moe {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = kSampleThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 9, kBins = 1 << kBinBits;
static_assert(kBins == kThreads, "a thread looks at one bin");
constexpr int kList = 128;
constexpr int kMassBits = 42;
static_assert(kList * 4 <= kThreads, "four threads rank a member");

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// (.aligned asks for whole warps: what comes before is often one lane's)
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// (the two halves by themselves at the start: shared memory of a CTA that has
// not begun may not be written)
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// The address of this CTA's shared variable in CTA r of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t r) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(r));
    return a;
}
__device__ __forceinline__ u64 ld_remote64(uint32_t a) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_remote64(uint32_t a, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void st_remote32(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t atom_add_remote32(uint32_t a, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(a), "r"(v) : "memory");
    return old;
}

struct Shared {
    // a histogram: members of each bin, and the sum of their places in it or of
    // their masses; and the same over the cluster
    struct {
        uint32_t count[kBins];
        union {
            uint32_t place[kBins];
            u64 mass[kBins];
        };
    } hist, all;
    struct {  // members of the border's bin (first CTA of the cluster)
        u64 code[kList];
        u64 mass[kList];
        uint32_t index[kList];
        uint16_t order[kList];
        u64 sums[kList];
    } list;
    uint16_t queue[kWarps][32 + 128];  // indices that a warp has put aside
    u64 best[16];       // each CTA's largest logit and its index
    // each CTA's share of a cluster sum, in two sets used in turn: a CTA that
    // is a barrier ahead writes the other set than the one still being read
    u64 part[2][16];
    u64 warp_sum[2][kWarps];
    // what the search for a border found
    u64 before, border;
    uint32_t bin_count, bin, bin_to, tie_limit;
    uint32_t listed;
};

// Ascending with the value; +0 and -0 were made one before.
__device__ __forceinline__ uint32_t value_bits(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float bits_value(uint32_t v) {
    return __uint_as_float(v ^ ((v >> 31) ? 0x80000000u : 0xffffffffu));
}

struct Scale {
    float top;      // the row's largest logit
    float hi, lo;   // log2(e) / T
};

// A logit's place: t in 2^-17 steps, monotone in x, since each of its three
// roundings is. From kNoPart on (t = 41, -inf) it has no part in the mass.
constexpr uint32_t kStepBits = 23, kNoPart = 41u << 17;
__device__ __forceinline__ uint32_t steps_of(float x, const Scale& s) {
    return __float_as_uint(__fmaf_rn(__fsub_rn(s.top, x), s.hi, 64.f)) - 0x42800000u;
}
// Its mass w in units of 2^-42, given that it has a part. Each operation rounds
// as it is written: were the product th fused into the sums that use it, its
// error would count twice there, and a mass would not have the bits that the
// paired form below gives it. (A row's total comes from the one and the search
// in a thread's logits from the other: they have to end at the same number.)
__device__ __forceinline__ u64 mass_of(float x, const Scale& s) {
    const float d = __fsub_rn(s.top, x);
    // the rounding error of the difference, then of the product
    const float bb = __fsub_rn(d, s.top), err = __fsub_rn(__fsub_rn(s.top, __fsub_rn(d, bb)), __fadd_rn(x, bb));
    const float th = __fmul_rn(d, s.hi);
    const float tl = __fadd_rn(__fmaf_rn(d, s.hi, -th), __fmaf_rn(d, s.lo, __fmul_rn(err, s.hi)));
    const float whole = __fadd_rn(th, 12582912.f);  // 1.5 * 2^23: rounds to a whole number n <= 41, in the low bits
    const uint32_t n = __float_as_uint(whole) & 0x3fu;
    const float f = __fadd_rn(__fsub_rn(th, __fsub_rn(whole, 12582912.f)), tl);
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-f));
    // e = mant * 2^(exponent - 150), the exponent 126 or 127
    const uint32_t b = __float_as_uint(e);
    const u64 mant = (u64)((b & 0x7fffffu) | 0x800000u) << (kMassBits - 23);
    return mant >> (n + 127u - (b >> 23));
}

// Both for two logits, with the paired fp32 operations: the same roundings, so
// the same bits.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus(float2 a, float2 b) { return ffma2(b, both(-1.f), a); }  // a - b
__device__ __forceinline__ void steps_of(float2 x, const Scale& s, uint32_t (&steps)[2]) {
    const float2 t = ffma2(minus(both(s.top), x), both(s.hi), both(64.f));
    steps[0] = __float_as_uint(t.x) - 0x42800000u;
    steps[1] = __float_as_uint(t.y) - 0x42800000u;
}
__device__ __forceinline__ void mass_of(float2 x, const Scale& s, u64 (&mass)[2]) {
    const float2 top = both(s.top), hi = both(s.hi), lo = both(s.lo), round = both(12582912.f);
    const float2 d = minus(top, x);
    const float2 bb = minus(d, top), err = minus(minus(top, minus(d, bb)), __fadd2_rn(x, bb));
    const float2 minus_t = __fmul2_rn(d, both(-s.hi));
    const float2 rest = __fadd2_rn(ffma2(d, hi, minus_t), ffma2(d, lo, __fmul2_rn(err, hi)));
    const float2 whole = minus(round, minus_t);
    const float2 minus_f = minus(__fadd2_rn(minus(whole, round), minus_t), rest);
    float e[2];
    asm("ex2.approx.f32 %0, %1;" : "=f"(e[0]) : "f"(minus_f.x));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e[1]) : "f"(minus_f.y));
    const uint32_t n[2] = {__float_as_uint(whole.x) & 0x3fu, __float_as_uint(whole.y) & 0x3fu};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t b = __float_as_uint(e[i]);
        mass[i] = ((u64)((b & 0x7fffffu) | 0x800000u) << (kMassBits - 23)) >> (n[i] + 127u - (b >> 23));
    }
}

// log2(e) / T as a sum of two fp32, without fp64 (two operations a clock and
// SM here: a division by every thread cost 10 us a call).
__device__ __forceinline__ void scale_of(float T, Scale& s) {
    constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f;  // their sum: log2(e) to 2^-48
    s.hi = fminf(__fdiv_rn(kLog2e, T), 1e30f);
    s.lo = s.hi < 1e30f ? __fdiv_rn(fmaf(-s.hi, T, kLog2e) + kLog2eRest, T) : 0.f;
    if (!(fabsf(s.lo) < 1e30f)) s.lo = 0.f;  // T = inf
}

// floor(f * v), or the next whole number above f * v, for 0 <= f < 1: the 24
// bits of f times v in 128 bits, shifted.
__device__ __forceinline__ u64 share(float f, u64 v, bool up) {
    const uint32_t b = __float_as_uint(f);
    const int e = (int)(b >> 23);
    const u64 mant = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int sh = 150 - (e ? e : 1);  // f = mant * 2^-sh, 24 <= sh < 150
    const u64 lo = mant * v, hi = __umul64hi(mant, v);
    u64 q, rest;
    if (sh < 64) {
        q = (hi << (64 - sh)) | (lo >> sh);
        rest = lo << (64 - sh);
    } else {
        q = sh < 128 ? (sh == 64 ? hi : hi >> (sh - 64)) : 0;
        rest = lo | (sh >= 128 ? hi : sh == 64 ? 0 : hi << (128 - sh));
    }
    return q + (up && rest ? 1 : 0);
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Shared memory of a CTA: Shared, then the slice.
__host__ __device__ constexpr int offset_slice() { return (int)((sizeof(Shared) + 15) & ~size_t(15)); }

// A member into the histogram of all codes: its bin is an eighth of a unit of t.
__device__ __forceinline__ void enter_bin(Shared& sh, uint32_t steps) {
    const uint32_t bin = steps >> (kStepBits - kBinBits);
    atomicAdd(&sh.hist.count[bin], 1u);
    atomicAdd(&sh.hist.place[bin], (steps >> (kStepBits - kBinBits - 8)) & 255u);
}

// The row's slice that this CTA holds, and what bounds the kept set so far:
// steps below `limit`, codes up to `border`, of those equal to it the indices
// up to `tie`.
struct Row {
    const float* x;
    int n, base;  // logits and first index
    int len;      // logits of a thread
    Scale scale;
    uint32_t limit;
    u64 border;
    uint32_t tie;
    int turn;  // which set of cluster sums is in use
};
constexpr int kCodeBits = kStepBits + 32;
__device__ __forceinline__ u64 code_of(uint32_t steps, float x) { return ((u64)steps << 32) | (uint32_t)~value_bits(x); }
// Steps below this are kept for certain: the border's own are limit - 1.
__device__ __forceinline__ uint32_t sure_steps(const Row& r) { return r.border == ~0ull ? r.limit : r.limit - 1; }
__device__ __forceinline__ bool kept(const Row& r, u64 code, uint32_t index) {
    return code < r.border || (code == r.border && index <= r.tie);
}
// Each thread takes consecutive logits, an odd number of 16-byte words so that
// eight lanes' words lie in all the banks; the slice is filled up with -inf to
// a whole number of threads.
__host__ __device__ __forceinline__ int per_thread(int n) { return (((n + 4 * kThreads - 1) / (4 * kThreads)) | 1) * 4; }

// The mass of the thread's logits with steps in [from, to); f(i, x, steps) for
// those with steps in [to, row.limit), in the thread itself (OWN) or in any of
// its warp. COUNT: each of the former also goes into the histogram, into its
// bin's number of members and the sum of their places within the bin. The
// masses of four are taken together, without a branch between them: one's chain
// is some 30 operations. The others are few, but hardly any 128 logits have
// none, so they are queued and taken 32 at a time.
template <bool COUNT, bool OWN, class F>
__device__ __forceinline__ u64 sweep(const Row& row, uint32_t from, uint32_t to, Shared& sh, F f) {
    const int lane = threadIdx.x & 31;
    const int i0 = threadIdx.x * row.len, i1 = i0 + row.len;
    const uint32_t span = to > from ? to - from : 0, few = row.limit > to ? row.limit - to : 0;
    uint16_t* queue = sh.queue[threadIdx.x >> 5];
    int queued = 0;
    auto flush = [&] {
        __syncwarp();
        for (int n = lane; n < queued; n += 32) {
            const int i = queue[n];
            f(i, row.x[i], steps_of(row.x[i], row.scale));
        }
        __syncwarp();
        queued = 0;
    };
    u64 sum = 0;
    for (int i = i0; i < i1; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(row.x + i);
        const float x[4] = {q.x, q.y, q.z, q.w};
        uint32_t steps[4], two[2];
        steps_of(make_float2(q.x, q.y), row.scale, two);
        steps[0] = two[0], steps[1] = two[1];
        steps_of(make_float2(q.z, q.w), row.scale, two);
        steps[2] = two[0], steps[3] = two[1];
        bool in = false, near = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            in |= steps[j] - from < span;
            near |= steps[j] - to < few;
        }
        if (in) {
            u64 w[4], pair[2];
            mass_of(make_float2(q.x, q.y), row.scale, pair);
            w[0] = pair[0], w[1] = pair[1];
            mass_of(make_float2(q.z, q.w), row.scale, pair);
            w[2] = pair[0], w[3] = pair[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum += steps[j] - from < span ? w[j] : 0;
                if (COUNT && steps[j] - from < span) enter_bin(sh, steps[j]);
            }
        }
        if (OWN) {
            if (near) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (steps[j] - to < few) f(i + j, x[j], steps[j]);
            }
        } else if (__any_sync(0xffffffffu, near)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool one = steps[j] - to < few;
                const uint32_t set = __ballot_sync(0xffffffffu, one);
                if (one) queue[queued + __popc(set & ((1u << lane) - 1u))] = (uint16_t)(i + j);
                queued += __popc(set);
            }
            if (queued >= 32) flush();
        }
    }
    if (!OWN) flush();
    return sum;
}
// A run of 2^width codes from `from` on.
struct Range {
    u64 from;
    int width;
    int shift;  // codes of a bin, as a power of two
    __device__ __forceinline__ bool has(u64 code) const { return ((code - from) >> width) == 0; }
    __device__ __forceinline__ uint32_t bin(u64 code) const { return (uint32_t)((code - from) >> shift); }
    __device__ __forceinline__ void split() { shift = max(width - kBinBits, 0); }
};

enum Search { kByCount, kByMass, kByBounds };

// The bin of the cluster's histogram in which the target is reached: in
// sh.bin_count (0: it is not reached), sh.bin and, with what lies before the
// bin, sh.before. `own` is summed over the threads and added to
// `all`. kByMass starts from `all`. kByBounds takes `part` of `all` as the
// target, and finds the first bin in which the bins' largest possible masses
// reach it and the first (sh.bin_to) in which their smallest do.
template <Search S>
__device__ __forceinline__ void locate(Row& row, u64& target, float part, u64 own, u64& all, Shared& sh, uint32_t rank,
                                       int C) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    own = warp_sum(own);
    if (lane == 0) sh.warp_sum[0][warp] = own;
    if (tid == 0) {
        sh.bin_count = 0;
        sh.bin_to = kBins - 1;
        // (here, before a barrier of the cluster: what follows may append to the
        // first CTA's list at once)
        sh.listed = 0;
    }
    __syncthreads();
    if (tid < C) {
        u64 a = 0;
        for (int w = 0; w < kWarps; ++w) a += sh.warp_sum[0][w];
        st_remote64(remote(&sh.part[row.turn][rank], tid), a);
    }
    cluster_sync();
    // Each CTA sums 512 / C bins and leaves the sums in all CTAs: a thread reads
    // one bin of one CTA and writes one sum to one. (With masses and C = 16 all of
    // this takes 10,500 cycles, and 14,200 where every CTA reads all of the
    // others' bins; the wait for the slowest CTA's sweep is in both.)
    {
        const int r = tid & (C - 1), bin = (int)rank * (kBins / C) + tid / C;
        uint32_t n = ld_remote32(remote(&sh.hist.count[bin], r));
        u64 v = S == kByMass     ? ld_remote64(remote(&sh.hist.mass[bin], r))
                : S == kByBounds ? ld_remote32(remote(&sh.hist.place[bin], r))
                                 : 0;
        for (int o = C / 2; o; o >>= 1) {
            n += __shfl_xor_sync(0xffffffffu, n, o);
            if (S != kByCount) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        st_remote32(remote(&sh.all.count[bin], r), n);
        if (S == kByMass) st_remote64(remote(&sh.all.mass[bin], r), v);
        if (S == kByBounds) st_remote32(remote(&sh.all.place[bin], r), (uint32_t)v);
    }
    cluster_sync();
    const uint32_t count = sh.all.count[tid];
    const u64 value = S == kByMass ? sh.all.mass[tid] : S == kByBounds ? sh.all.place[tid] : 0;
    for (int r = 0; r < C; ++r) all += sh.part[row.turn][r];
    if (S == kByBounds) {
        target = part > 0.f ? share(part, all, true) : 0;
        target = target > 1 ? target : 1;
    }
    u64 sum[2] = {S == kByMass ? value : count, 0};  // what is searched; kByBounds: largest, smallest
    if (S == kByBounds) {
        sum[0] = 0;
        if (count) {
            // The mean of t, in parts of the bin, is known to 1/256. The mass
            // of one falls from `first` to `first` 2^(-1/8) within the bin and
            // is convex in t, so the mean mass is at least that of the mean t
            // and at most the chord's there. 2^-16: t is off by its rounding; 1:
            // a mass is cut to whole units.
            const float first = exp2f((float)kMassBits - (float)tid * (1.f / 8.f));
            const float mean = (float)value / ((float)count * 256.f);
            const float most = first * (1.f - 0.08299595f * mean) * (1.f + 1.f / 65536.f);
            const float least = first * exp2f((mean + 1.f / 256.f) * (-1.f / 8.f)) * (1.f - 1.f / 65536.f);
            sum[0] = count * __float2ull_ru(most);
            sum[1] = least > 1.f ? count * (__float2ull_rd(least) - 1) : 0;
        }
    }
    u64 upto[2] = {sum[0], sum[1]};
#pragma unroll
    for (int k = 0; k < (S == kByBounds ? 2 : 1); ++k) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 a = __shfl_up_sync(0xffffffffu, upto[k], o);
            if (lane >= o) upto[k] += a;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.warp_sum[0][warp] = upto[0];
        sh.warp_sum[1][warp] = upto[1];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (S == kByBounds ? 2 : 1); ++k) {
        u64 before = (S == kByMass ? all : 0) + upto[k] - sum[k];
        for (int w = 0; w < warp; ++w) before += sh.warp_sum[k][w];
        if (before < target && target <= before + sum[k]) {
            if (k == 0) {
                sh.bin = tid;
                sh.bin_count = count;
                sh.before = before;
            } else {
                sh.bin_to = tid;
            }
        }
    }
    __syncthreads();
}

// Gathers the range's members in the first CTA, which ranks them and finds the
// last one that is kept: the count-th (0: the last of all) and, with by_mass,
// the first up to which the mass reaches `goal`, or where that is 0 `part` of
// the mass up to the count-th. False when there are more than kList. WITH_BELOW:
// the goal counts from the first of all; the thread's mass before the range
// (which begins with a step) is left in `below`.
template <bool WITH_BELOW>
__device__ __forceinline__ bool settle(Row& row, const Range range, u64 count, bool by_mass, u64 goal, float part,
                                       u64& below, Shared& sh, uint32_t rank, int C) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t first = (uint32_t)(range.from >> 32);
    const u64 own = sweep<false, false>(row, WITH_BELOW ? 0 : first, first, sh, [&](int i, float x, uint32_t steps) {
        const u64 code = code_of(steps, x);
        if (!range.has(code) || !kept(row, code, row.base + i)) return;
        const uint32_t at = atom_add_remote32(remote(&sh.listed, 0), 1u);
        if (at < kList) {
            st_remote64(remote(&sh.list.code[at], 0), code);
            st_remote64(remote(&sh.list.mass[at], 0), mass_of(x, row.scale));
            st_remote32(remote(&sh.list.index[at], 0), row.base + i);
        }
    });
    if (WITH_BELOW) {
        below = own;
        const u64 sum = warp_sum(own);
        if (lane == 0) sh.warp_sum[0][warp] = sum;
        __syncthreads();
        if (tid == 0) {
            u64 all = 0;
            for (int w = 0; w < kWarps; ++w) all += sh.warp_sum[0][w];
            st_remote64(remote(&sh.part[row.turn][rank], 0), all);
        }
    }
    cluster_sync();
    if (WITH_BELOW)
        for (int r = 0; r < C; ++r) goal -= sh.part[row.turn][r];  // (the first CTA's alone is used)
    const uint32_t members = ld_remote32(remote(&sh.listed, 0));
    const bool fits = members <= kList;
    if (rank == 0 && fits) {
        // four threads or more count the members before one
        {
            const int team = members <= 32 ? 16 : members <= 64 ? 8 : 4;
            const uint32_t i = tid / team;
            uint32_t place = 0;
            if (i < members) {
                const u64 code = sh.list.code[i];
                const uint32_t index = sh.list.index[i];
                for (uint32_t j = tid & (team - 1); j < members; j += team) {
                    const u64 other = sh.list.code[j];
                    place += other < code || (other == code && sh.list.index[j] < index);
                }
            }
            for (int o = team / 2; o; o >>= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
            if (i < members && (tid & (team - 1)) == 0) sh.list.order[place] = (uint16_t)i;
        }
        __syncthreads();
        // mass up to each place
        if (tid < kList) {
            const u64 own = (uint32_t)tid < members ? sh.list.mass[sh.list.order[tid]] : 0;
            u64 upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            if (lane == 31) sh.warp_sum[0][warp] = upto;
            __syncwarp();
            named_bar_sync(1, kList);
            for (int w = 0; w < warp; ++w) upto += sh.warp_sum[0][w];
            sh.list.sums[tid] = upto;
            named_bar_sync(1, kList);
            const uint32_t last = (count ? (uint32_t)min(count, (u64)members) : members) - 1;
            if (by_mass && goal == 0) {
                goal = part > 0.f ? share(part, sh.list.sums[last], true) : 0;
                goal = goal > 1 ? goal : 1;
            }
            const bool here = by_mass && goal <= sh.list.sums[last] ? upto - own < goal && goal <= upto : tid == (int)last;
            if ((uint32_t)tid < members && here) {
                sh.border = sh.list.code[sh.list.order[tid]];
                sh.tie_limit = sh.list.index[sh.list.order[tid]];
            }
        }
    }
    cluster_sync();
    if (fits) {
        row.border = ld_remote64(remote(&sh.border, 0));
        row.tie = ld_remote32(remote(&sh.tie_limit, 0));
        row.limit = min(row.limit, (uint32_t)(row.border >> 32) + 1);
        cluster_sync();
    }
    return fits;
}

// Narrows the row to its first k members (k > 0), and of those to the shortest
// run that reaches `part` of their mass (by_p). `top` is the thread's largest
// logit. The mass of the thread's logits with steps below `summed`, all of
// them kept, is left in `below`.
__device__ __forceinline__ void narrow(Row& row, int k, bool by_p, float part, float top, uint32_t& summed, u64& below,
                                       Shared& sh, uint32_t rank, int C) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto clear = [&] {
        row.turn ^= 1;
        for (int i = tid; i < kBins; i += kThreads) {
            sh.hist.count[i] = 0;
            sh.hist.mass[i] = 0;  // (and so the places)
        }
        __syncthreads();
    };
    for (int stage = k > 0 ? 0 : 1; stage < (by_p ? 2 : 1); ++stage) {
        const bool by_mass = stage == 1;
        u64 target = (u64)k, all = 0;
        Range range = {0, kCodeBits, kCodeBits - kBinBits};
        clear();
        if (!by_mass) {
            const uint32_t steps = steps_of(top, row.scale);
            if (steps < row.limit) atomicAdd(&sh.hist.count[range.bin(code_of(steps, top))], 1u);
            locate<kByCount>(row, target, 0.f, 0, all, sh, rank, C);
            if (sh.bin_count) {
                row.limit = min(row.limit, (sh.bin + 1) << (kStepBits - kBinBits));
                if (k <= kList && settle<false>(row, range, (u64)k, by_p, 0, part, below, sh, rank, C)) return;
            }
            clear();
        } else {
            u64 near = 0;
            u64 own = sweep<true, true>(row, 0, sure_steps(row), sh, [&](int i, float x, uint32_t steps) {
                if (!kept(row, code_of(steps, x), row.base + i)) return;
                near += mass_of(x, row.scale);
                enter_bin(sh, steps);
            });
            own += near;
            locate<kByBounds>(row, target, part, own, all, sh, rank, C);
            const uint32_t b1 = sh.bin, b2 = sh.bin_to;
            range.width = kCodeBits - kBinBits + (b2 > b1 ? 32 - __clz((int)(b2 - b1)) : 0);
            range.from = (u64)b1 << (kCodeBits - kBinBits);
            row.limit = min(row.limit, (b2 + 1) << (kStepBits - kBinBits));
            summed = b1 << (kStepBits - kBinBits);
            all = 0;
            // few members there (a row with some likely tokens): ranked at once
            uint32_t members = kList + 1;
            if (b2 - b1 < 16) {
                members = 0;
                for (uint32_t b = b1; b <= b2; ++b) members += sh.all.count[b];
            }
            clear();
            if (members <= kList) {
                settle<true>(row, range, 0, true, target, 0.f, below, sh, rank, C);
                return;
            }
        }
        for (bool again = false;; again = true) {
            range.split();
            const int shift = range.shift;
            auto enter = [&](int i, float x, uint32_t steps) {
                const u64 code = code_of(steps, x);
                if (!range.has(code) || !kept(row, code, row.base + i)) return;
                const uint32_t at = range.bin(code);
                atomicAdd(&sh.hist.count[at], 1u);
                if (by_mass) atomicAdd(&sh.hist.mass[at], mass_of(x, row.scale));
            };
            const uint32_t first = (uint32_t)(range.from >> 32);
            const u64 own = sweep<false, false>(row, by_mass && !again ? 0 : first, first, sh, enter);
            if (by_mass && !again) below = own;
            if (by_mass) locate<kByMass>(row, target, 0.f, own, all, sh, rank, C);
            else locate<kByCount>(row, target, 0.f, 0, all, sh, rank, C);
            const uint32_t members = sh.bin_count, bin = sh.bin;
            if (members == 0) break;  // fewer than k: all are kept
            if (!by_mass) target -= sh.before;
            range.from += (u64)bin << shift;
            range.width = shift;
            if (by_mass ? members == 1 : target == members) {  // all of the bin is kept
                const u64 bound = range.from + ((1ull << shift) - 1ull);
                if (bound < row.border) {
                    row.border = bound;
                    row.tie = 0xffffffffu;
                    row.limit = min(row.limit, (uint32_t)(bound >> 32) + 1);
                }
                break;
            }
            const u64 rest = by_mass ? target - sh.before : target;
            if (members <= kList) {
                settle<false>(row, range, by_mass ? 0 : rest, by_mass, rest, 0.f, below, sh, rank, C);
                break;
            }
            if (shift == 0) {
                // more than kList members of one value: all of one mass, in
                // index order
                const u64 each = mass_of(bits_value(~(uint32_t)range.from), row.scale);
                const u64 need = by_mass ? (rest + each - 1) / each : rest;
                const uint32_t mine = sh.hist.count[bin];
                uint32_t lower = 0;
                for (uint32_t r = 0; r < rank; ++r) lower += ld_remote32(remote(&sh.hist.count[bin], r));
                if (lower < need && need <= (u64)lower + mine) {
                    // thread by thread, as they lie
                    const int i0 = min(tid * row.len, row.n), i1 = min(i0 + row.len, row.n);
                    auto tied = [&](int i) {
                        const u64 code = code_of(steps_of(row.x[i], row.scale), row.x[i]);
                        return code == range.from && kept(row, code, row.base + i);
                    };
                    uint32_t n = 0;
                    for (int i = i0; i < i1; ++i) n += tied(i);
                    uint32_t upto = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                        if (lane >= o) upto += v;
                    }
                    __syncthreads();
                    if (lane == 31) sh.warp_sum[0][warp] = upto;
                    __syncthreads();
                    u64 place = (u64)lower + upto - n;
                    for (int w = 0; w < warp; ++w) place += sh.warp_sum[0][w];
                    if (place < need && need <= place + n) {
                        int i = i0;
                        for (;; ++i)
                            if (tied(i) && ++place == need) break;
                        for (int r = 0; r < C; ++r) st_remote32(remote(&sh.tie_limit, r), row.base + i);
                    }
                }
                cluster_sync();
                row.border = range.from;
                row.tie = sh.tie_limit;
                row.limit = min(row.limit, (uint32_t)(row.border >> 32) + 1);
                cluster_sync();
                break;
            }
            all = sh.before;
            __syncthreads();  // all have read what was found
            clear();
        }
    }
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    float x = DT == 0 ? static_cast<const float*>(p)[i]
                      : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return x;
}
// NaN counts as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY) + 0.f; }

// The most shared memory of a CTA: the longest slice fills 23 words of 16 bytes
// a thread.
constexpr int kSampleSmem = offset_slice() + 23 * 16 * kThreads;
static_assert(kSampleSmem <= 232448 && kSampleMaxSlice <= 22 * 4 * kThreads, "shared memory of a CTA");
constexpr size_t kSampleSmemOfTwo = 113 * 1024;

template <int DT>
__global__ __launch_bounds__(kThreads, 2) void sample_kernel(SampleParams p) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared& sh = *reinterpret_cast<Shared*>(dyn);
    float* xs = reinterpret_cast<float*>(dyn + offset_slice());
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int C = p.C, m = blockIdx.x / C;
    cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    // (asked for before the logits: each would otherwise be waited for on its own)
    const float T = p.temperature ? p.temperature[m] : 1.f;
    const int k = p.top_k ? p.top_k[m] : 0;
    const float top_p = p.top_p ? p.top_p[m] : 1.f;
    const float min_p = p.min_p ? p.min_p[m] : 0.f;
    const float u = p.u[m];

    Row row;
    row.base = (int)rank * p.slice;
    row.n = max(0, min(p.slice, p.V - row.base));
    row.x = xs;
    row.len = per_thread(p.slice);
    row.border = ~0ull;
    row.tie = 0xffffffffu;
    row.limit = kNoPart;
    row.turn = 0;
    // the slice into shared memory; its largest logit, lowest index first
    const int64_t start = (int64_t)m * p.row_stride + row.base;
    float own_top = -INFINITY;
    int own_at = 0;
    auto see = [&](float x, int i) {  // (a thread's indices ascend)
        xs[i] = x;
        if (x > own_top) {
            own_top = x;
            own_at = i;
        }
    };
    const uint8_t* src = static_cast<const uint8_t*>(p.logits) + start * (DT == 0 ? 4 : 2);
    constexpr int kVec = DT == 0 ? 4 : 8;
    const int nv = (reinterpret_cast<uintptr_t>(src) & 15u) == 0 ? row.n / kVec : 0;
    for (int v0 = tid; v0 < nv; v0 += 4 * kThreads) {
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v0 + j * kThreads < nv) q[j] = reinterpret_cast<const uint4*>(src)[v0 + j * kThreads];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int v = v0 + j * kThreads;
            if (v >= nv) break;
            if (DT == 0) {
                see(clean(__uint_as_float(q[j].x)), v * kVec);
                see(clean(__uint_as_float(q[j].y)), v * kVec + 1);
                see(clean(__uint_as_float(q[j].z)), v * kVec + 2);
                see(clean(__uint_as_float(q[j].w)), v * kVec + 3);
            } else {
                float f[8];
                unpack8(q[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) see(clean(f[e]), v * kVec + e);
            }
        }
    }
    for (int i = nv * kVec + tid; i < row.n; i += kThreads) see(clean(load_logit<DT>(src, i)), i);
    for (int i = row.n + tid; i < row.len * kThreads; i += kThreads) xs[i] = -INFINITY;
    u64 best = row.n > 0 ? ((u64)value_bits(own_top) << 32) | (uint32_t)~(uint32_t)(row.base + own_at) : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
    }
    if (lane == 0) sh.warp_sum[0][warp] = best;
    cluster_wait();
    __syncthreads();
    if (tid < C) {
        for (int w = 0; w < kWarps; ++w) best = sh.warp_sum[0][w] > best ? sh.warp_sum[0][w] : best;
        st_remote64(remote(&sh.best[rank], tid), best);
    }
    cluster_sync();
    best = 0;
    for (int r = 0; r < C; ++r) best = sh.best[r] > best ? sh.best[r] : best;
    row.scale.top = bits_value((uint32_t)(best >> 32));
    const bool none = !(row.scale.top > -INFINITY);
    if (none || !(T > 0.f) || k == 1) {
        if (rank == 0 && tid == 0) {
            p.token[m] = none ? -1 : (int)~(uint32_t)best;
            if (p.prob) p.prob[m] = none ? 0.f : 1.f;
        }
        return;  // no CTA reads another's memory after the last barrier
    }
    scale_of(T, row.scale);

    const bool by_p = top_p < 1.f;
    if (row.scale.top == INFINITY) {
        // infinities share the mass: equal logits before nothing
        for (int i = tid; i < row.n; i += kThreads) xs[i] = xs[i] == INFINITY ? 0.f : -INFINITY;
        own_top = own_top == INFINITY ? 0.f : -INFINITY;
        row.scale.top = 0.f;
        __syncthreads();
    }
    uint32_t summed = 0;
    u64 below = 0;
    if ((k > 0 && k < p.V) || by_p) narrow(row, k < p.V ? max(k, 0) : 0, by_p, top_p, own_top, summed, below, sh, rank, C);

    // The kept mass in index order. Whether w >= min_p is asked only where t
    // is within 2^-10 of -log2(min_p).
    uint32_t sure = sure_steps(row);
    u64 least = 0;
    if (min_p > 0.f) {
        const float ratio = fminf(min_p, 1.f);
        least = __float2ull_ru(ratio * (float)(1ull << kMassBits));
        const uint32_t t = (uint32_t)(fminf(-log2f(ratio), 41.f) * (float)(1 << (kStepBits - 6)));
        sure = min(sure, t > 128 ? t - 128 : 0);
        row.limit = min(row.limit, t + 129);
    }
    auto mass_at = [&](int i, float x, uint32_t steps) -> u64 {
        if (steps >= row.limit || !kept(row, code_of(steps, x), row.base + i)) return 0;
        const u64 w = mass_of(x, row.scale);
        return w >= least ? w : 0;
    };
    u64 near = 0;
    const uint32_t from = summed <= sure ? summed : 0;
    u64 own = sweep<false, true>(row, from, sure, sh, [&](int i, float x, uint32_t steps) { near += mass_at(i, x, steps); });
    own += near + (from ? below : 0);
    const int i0 = min(tid * row.len, row.n), i1 = min(i0 + row.len, row.n);
    u64 upto = own;  // of the warp's threads up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sum[0][warp] = upto;
    __syncthreads();
    row.turn ^= 1;
    if (tid < C) {
        u64 sum = 0;
        for (int i = 0; i < kWarps; ++i) sum += sh.warp_sum[0][i];
        st_remote64(remote(&sh.part[row.turn][rank], tid), sum);
    }
    cluster_sync();
    u64 before = 0, all = 0;
    for (int r = 0; r < C; ++r) {
        if (r < (int)rank) before += sh.part[row.turn][r];
        all += sh.part[row.turn][r];
    }
    for (int i = 0; i < warp; ++i) before += sh.warp_sum[0][i];
    const u64 goal = !(u > 0.f) ? 0ull : u < 1.f ? share(u, all, false) : all - 1;
    // the thread whose logits hold the first cumulated mass above the goal,
    // then its warp over those logits
    before += upto - own;
    const uint32_t holder = __ballot_sync(0xffffffffu, before <= goal && goal < before + own);
    if (holder == 0) return;
    const int who = __ffs(holder) - 1;
    before = __shfl_sync(0xffffffffu, before, who);
    const int begin = __shfl_sync(0xffffffffu, i0, who), to = __shfl_sync(0xffffffffu, i1, who);
    for (int i = begin; i < to; i += 32) {
        const u64 one = i + lane < to ? mass_at(i + lane, xs[i + lane], steps_of(xs[i + lane], row.scale)) : 0ull;
        u64 sum = one;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (before + sum - one <= goal && goal < before + sum) {
            p.token[m] = row.base + i + lane;
            if (p.prob) p.prob[m] = __fdiv_rn(__ull2float_rn(one), __ull2float_rn(all));
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        if (before > goal) break;
    }
}

}  // namespace

// CTAs a row. Rows that can all be on the GPU at once are spread over as many
// CTAs as can (a cluster of 8 of one CTA an SM fits 15 times on a GB300, of two
// an SM 36 times: 16 rows of 157,184 logits without filters took 20.1 us when
// the 16th had to wait, 17.0 then), each with at least 2,048 logits; more rows
// in slices of which two fit an SM.
cudaError_t launch_sample(SampleParams p, int M, int dtype, cudaStream_t stream) {
    void (*kern)(SampleParams) = dtype == 0 ? sample_kernel<0> : sample_kernel<1>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSampleSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    auto shape = [&](int C) {
        p.C = C;
        p.slice = ((p.V + C - 1) / C + 7) / 8 * 8;
        cfg.dynamicSmemBytes = (size_t)offset_slice() + (size_t)per_thread(p.slice) * kThreads * 4;
        attr[0].val.clusterDim.x = (unsigned)C;
        cfg.gridDim = dim3((unsigned)((int64_t)M * C));
        return p.slice <= kSampleMaxSlice;
    };
    // 1 + the clusters of 2^i CTAs, j + 1 CTAs an SM (the kernel's registers
    // allow no more), that are on this GPU at once (asked once; 0: not yet)
    static std::atomic<int> active[kMaxDevices][2][5][2];
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    int best = 0;
    for (int i = 4; i >= 0 && best == 0; --i) {
        if (!shape(1 << i) || (i > 0 && p.V / (1 << i) < 2048)) continue;
        std::atomic<int>& known = active[dev][dtype == 0 ? 0 : 1][i][cfg.dynamicSmemBytes <= kSampleSmemOfTwo ? 1 : 0];
        int n = known.load(std::memory_order_relaxed) - 1;
        if (n < 0) {
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
            if (e != cudaSuccess) return e;
            known.store(n + 1, std::memory_order_relaxed);
        }
        if (M <= n) best = 1 << i;
    }
    for (int C = 1; C <= 16 && best == 0; C *= 2)
        if (shape(C) && (cfg.dynamicSmemBytes <= kSampleSmemOfTwo || C == 16)) best = C;
    shape(best);
    // (a grid's limit, which no logits in memory reach)
    if ((int64_t)M * best > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe
