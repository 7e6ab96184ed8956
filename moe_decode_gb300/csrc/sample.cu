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
// descending, index ascending), encoded in 64 bits as (t in 2^-26 steps, the
// bits of l reversed); top-k and top-p each look for the last member by a
// histogram of 2048 bins of that code (count and mass), summed across the
// cluster through distributed shared memory. The bin that holds the border is
// split again, or, once it has at most kList members, gathered by the first
// CTA and ranked directly.
#include "paged.h"
#include "ptx.cuh"

namespace moe {
namespace {

using u64 = unsigned long long;
constexpr int kThreads = kSampleThreads;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kSampleBins;
constexpr int kList = 128;
constexpr int kMassBits = 42;
static_assert(kList * 4 == kThreads, "four threads rank a member");

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
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
    union {
        struct {
            u64 mass[kBins];
            uint32_t count[kBins];
        } hist;
        struct {  // members of the border's bin (first CTA of the cluster)
            u64 code[kList];
            u64 mass[kList];
            uint32_t index[kList];
            uint16_t order[kList];
        } list;
    };
    u64 best[16];       // each CTA's largest logit and its index
    // each CTA's share of a cluster sum, in two sets used in turn: a CTA that
    // is a barrier ahead writes the other set than the one still being read
    u64 part_mass[2][16];
    uint32_t part_count[2][16];
    u64 warp_mass[kWarps];
    u64 warp_count[kWarps];
    // what the search for a border found
    u64 before_mass, bin_mass, border;
    uint32_t before_count, bin_count, bin, tie_limit;
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

// t in 2^-26 steps (0xffffffff from 64 on: no mass); monotone in x, since
// each of the two roundings is.
__device__ __forceinline__ uint32_t steps_below(float x, const Scale& s) {
    const float d = x == s.top ? 0.f : s.top - x;
    const float t = d * s.hi;
    return d < 3.0e38f && t < 64.f ? (uint32_t)(t * 67108864.f) : 0xffffffffu;
}

// w in units of 2^-42.
__device__ __forceinline__ u64 mass_of(float x, const Scale& s) {
    if (x == s.top) return 1ull << kMassBits;
    const float d = s.top - x;
    if (!(d < 3.0e38f)) return 0;
    // the rounding error of the difference, then of the product
    const float bb = d - s.top, err = (s.top - (d - bb)) - (x + bb);
    const float th = d * s.hi;
    if (!(th < 43.5f)) return 0;
    const float tl = fmaf(d, s.hi, -th) + fmaf(d, s.lo, err * s.hi);
    const float n = rintf(th);
    const float f = (th - n) + tl;
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(-f));
    const u64 mant = (u64)__float2uint_rn(e * 16777216.f);
    const int sh = kMassBits - 24 - (int)n;
    return sh >= 0 ? mant << sh : (mant + (1ull << (-sh - 1))) >> -sh;
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Shared memory of a CTA: Shared, then the sums over the cluster of the bins
// that the CTA owns (clusters of two or more; a single CTA's histogram is the
// sum), then the slice.
__host__ __device__ constexpr int owned_bins(int C) { return C > 1 ? kBins / C : 0; }
__host__ __device__ constexpr int offset_sums() { return (int)((sizeof(Shared) + 15) & ~size_t(15)); }
__host__ __device__ constexpr int offset_slice(int C) { return offset_sums() + owned_bins(C) * 12; }
static_assert(offset_slice(16) % 16 == 0, "alignment of the slice");

// The row's slice that this CTA holds, and the bound of the kept set so far:
// codes up to `border`, of those equal to it the indices up to `tie`.
struct Row {
    const float* x;
    int n, base;  // members and first index
    Scale scale;
    u64 border;
    uint32_t tie;
    int turn;  // which set of cluster sums is next
};
__device__ __forceinline__ u64 code_of(uint32_t steps, float x) { return ((u64)steps << 32) | (uint32_t)~value_bits(x); }
__device__ __forceinline__ bool kept(const Row& r, u64 code, uint32_t index) {
    return code < r.border || (code == r.border && index <= r.tie);
}

// Narrows row.border to the last member of the kept set's shortest prefix
// whose count (BY_MASS false) or mass (true) reaches `target`; the set stays
// as it is where all of it does not. Returns the kept set's mass then
// (WITH_MASS: also kept by count searches).
template <bool BY_MASS>
__device__ u64 narrow(Row& row, u64 target, bool with_mass, Shared& sh, uint32_t rank, int C) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int own = kBins / C;  // bins that this CTA sums
    u64* red_mass = reinterpret_cast<u64*>(reinterpret_cast<uint8_t*>(&sh) + offset_sums());
    uint32_t* red_count = reinterpret_cast<uint32_t*>(red_mass + own);
    u64 before = 0;             // mass of the codes before the group
    u64 prefix = 0;
    int shift = 64;
    for (int level = 0; level < 6; ++level) {
        const int width = level == 2 || level == 5 ? 10 : 11, low = shift - width;
        for (int i = tid; i < kBins; i += kThreads) {
            sh.hist.mass[i] = 0;
            sh.hist.count[i] = 0;
        }
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        for (int i = tid; i < row.n; i += kThreads) {
            const float x = row.x[i];
            const uint32_t steps = steps_below(x, row.scale);
            if (steps == 0xffffffffu) continue;
            const u64 code = code_of(steps, x);
            if (level && (code >> shift) != prefix) continue;
            if (!kept(row, code, row.base + i)) continue;
            const u64 w = mass_of(x, row.scale);
            if (w == 0) continue;
            const uint32_t bin = (uint32_t)(code >> low) & ((1u << width) - 1u);
            atomicAdd(&sh.hist.count[bin], 1u);
            if (with_mass) atomicAdd(&sh.hist.mass[bin], w);
        }
        const u64* mass = sh.hist.mass;
        const uint32_t* count = sh.hist.count;
        uint32_t from = 0;
        u64 skipped_mass = 0;
        u64 skipped_count = 0;
        uint32_t mass_at = 0, count_at = 0;
        if (C > 1) {
            cluster_sync();
            u64 pm = 0;
            u64 pc = 0;
            for (int i = tid; i < own; i += kThreads) {
                u64 m = 0;
                uint32_t c = 0;
                for (int r = 0; r < C; ++r) {
                    c += ld_remote32(remote(&sh.hist.count[rank * own + i], r));
                    if (with_mass) m += ld_remote64(remote(&sh.hist.mass[rank * own + i], r));
                }
                red_mass[i] = m;
                red_count[i] = c;
                pm += m;
                pc += c;
            }
            pm = warp_sum(pm);
            pc = warp_sum(pc);
            if (lane == 0) {
                sh.warp_mass[warp] = pm;
                sh.warp_count[warp] = pc;
            }
            __syncthreads();
            row.turn ^= 1;
            if (tid < C) {
                u64 m = 0, c = 0;
                for (int w = 0; w < kWarps; ++w) {
                    m += sh.warp_mass[w];
                    c += sh.warp_count[w];
                }
                st_remote64(remote(&sh.part_mass[row.turn][rank], tid), m);
                st_remote32(remote(&sh.part_count[row.turn][rank], tid), (uint32_t)c);
            }
            cluster_sync();
            // the CTA whose bins hold the border
            int q = 0;
            for (; q < C - 1; ++q) {
                const u64 reach = BY_MASS ? skipped_mass + sh.part_mass[row.turn][q] : skipped_count + sh.part_count[row.turn][q];
                if (reach >= target) break;
                skipped_mass += sh.part_mass[row.turn][q];
                skipped_count += sh.part_count[row.turn][q];
            }
            from = (uint32_t)(q * own);
            mass_at = remote(red_mass, q);
            count_at = remote(red_count, q);
        } else {
            __syncthreads();
        }
        // the bin: each thread sums `per` of the owner's bins, a scan finds
        // the thread, the thread the bin
        const int per = (own + kThreads - 1) / kThreads;
        u64 m[4], sm = 0;
        uint32_t c[4];
        u64 sc = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = tid * per + j;
            m[j] = 0;
            c[j] = 0;
            if (j < per && i < own) {
                if (C > 1) {
                    c[j] = ld_remote32(count_at + 4u * i);
                    if (with_mass) m[j] = ld_remote64(mass_at + 8u * i);
                } else {
                    c[j] = count[i];
                    if (with_mass) m[j] = mass[i];
                }
            }
            sm += m[j];
            sc += c[j];
        }
        u64 im = sm, ic = sc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 a = __shfl_up_sync(0xffffffffu, im, o), b = __shfl_up_sync(0xffffffffu, ic, o);
            if (lane >= o) {
                im += a;
                ic += b;
            }
        }
        if (tid == 0) sh.bin_count = 0;
        __syncthreads();  // also: warp_mass was read
        if (lane == 31) {
            sh.warp_mass[warp] = im;
            sh.warp_count[warp] = ic;
        }
        __syncthreads();
        u64 bm = skipped_mass + im - sm, bc = skipped_count + ic - sc;
        for (int w = 0; w < warp; ++w) {
            bm += sh.warp_mass[w];
            bc += sh.warp_count[w];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u64 b = BY_MASS ? bm : bc, e = b + (BY_MASS ? m[j] : c[j]);
            if (c[j] && b < target && target <= e) {
                sh.bin = from + tid * per + j;
                sh.before_mass = bm;
                sh.before_count = (uint32_t)bc;
                sh.bin_mass = m[j];
                sh.bin_count = c[j];
            }
            bm += m[j];
            bc += c[j];
        }
        __syncthreads();
        const uint32_t members = sh.bin_count;
        if (members == 0) {  // all of the set does not reach the target (level 0 only)
            u64 total = 0;
            if (C > 1)
                for (int r = 0; r < C; ++r) total += sh.part_mass[row.turn][r];
            else
                for (int w = 0; w < kWarps; ++w) total += sh.warp_mass[w];
            __syncthreads();
            return total;
        }
        const uint32_t bin = sh.bin;
        const u64 bin_mass = sh.bin_mass, below = before + sh.before_mass;
        target -= BY_MASS ? sh.before_mass : sh.before_count;
        prefix = (prefix << width) | bin;
        shift = low;
        before = below;
        // all of the bin is kept
        if (BY_MASS ? members == 1 : target == members) {
            const u64 bound = shift == 0 ? prefix : (prefix << shift) | ((1ull << shift) - 1ull);
            if (bound < row.border) {
                row.border = bound;
                row.tie = 0xffffffffu;
            }
            __syncthreads();
            return before + bin_mass;
        }
        if (members <= kList) {
            // gather the bin's members in the first CTA and rank them
            __syncthreads();
            for (int i = tid; i < row.n; i += kThreads) {
                const float x = row.x[i];
                const uint32_t steps = steps_below(x, row.scale);
                if (steps == 0xffffffffu) continue;
                const u64 code = code_of(steps, x);
                if ((code >> shift) != prefix || !kept(row, code, row.base + i)) continue;
                const u64 w = mass_of(x, row.scale);
                if (w == 0) continue;
                const uint32_t at = atom_add_remote32(remote(&sh.listed, 0), 1u);
                st_remote64(remote(&sh.list.code[at], 0), code);
                st_remote64(remote(&sh.list.mass[at], 0), w);
                st_remote32(remote(&sh.list.index[at], 0), row.base + i);
            }
            cluster_sync();
            if (rank == 0) {
                // four threads count the members before one
                {
                    const uint32_t i = tid >> 2;
                    uint32_t place = 0;
                    if (i < members) {
                        const u64 code = sh.list.code[i];
                        const uint32_t index = sh.list.index[i];
                        for (uint32_t j = tid & 3; j < members; j += 4) {
                            const u64 other = sh.list.code[j];
                            place += other < code || (other == code && sh.list.index[j] < index);
                        }
                    }
                    place += __shfl_xor_sync(0xffffffffu, place, 1);
                    place += __shfl_xor_sync(0xffffffffu, place, 2);
                    if (i < members && (tid & 3) == 0) sh.list.order[place] = (uint16_t)i;
                }
                __syncthreads();
                // mass up to each place
                u64 own_mass = 0;
                if (tid < kList) {
                    own_mass = (uint32_t)tid < members ? sh.list.mass[sh.list.order[tid]] : 0;
                    u64 sum = own_mass;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const u64 v = __shfl_up_sync(0xffffffffu, sum, o);
                        if (lane >= o) sum += v;
                    }
                    if (lane == 31) sh.warp_mass[warp] = sum;
                    named_bar_sync(1, kList);
                    u64 b = sum - own_mass;
                    for (int w = 0; w < warp; ++w) b += sh.warp_mass[w];
                    const bool here = BY_MASS ? b < target && target <= b + own_mass : (u64)tid + 1 == target;
                    if ((uint32_t)tid < members && here) {
                        sh.border = sh.list.code[sh.list.order[tid]];
                        sh.tie_limit = sh.list.index[sh.list.order[tid]];
                        sh.bin_mass = b + own_mass;
                    }
                }
            }
            cluster_sync();
            row.border = ld_remote64(remote(&sh.border, 0));
            row.tie = ld_remote32(remote(&sh.tie_limit, 0));
            const u64 in_bin = ld_remote64(remote(&sh.bin_mass, 0));
            cluster_sync();
            return before + in_bin;
        }
    }
    // more than kList members of one value: all of one mass, in index order
    const u64 each = sh.bin_mass / sh.bin_count;
    const u64 need = BY_MASS ? (target + each - 1) / each : target;
    uint32_t mine = sh.hist.count[sh.bin], lower = 0;
    for (uint32_t r = 0; r < rank; ++r) lower += ld_remote32(remote(&sh.hist.count[sh.bin], r));
    if (lower < need && need <= (u64)lower + mine) {
        // warp by warp in index order
        const int chunk = ((row.n + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int i0 = warp * chunk, i1 = min(i0 + chunk, row.n);
        auto tied = [&](int i) {
            if (i >= i1) return false;
            const uint32_t steps = steps_below(row.x[i], row.scale);
            const u64 code = code_of(steps, row.x[i]);
            return code == prefix && kept(row, code, row.base + i);
        };
        uint32_t n = 0;
        for (int i = i0; i < i1; i += 32) n += __popc(__ballot_sync(0xffffffffu, tied(i + lane)));
        if (lane == 0) sh.warp_count[warp] = n;
        __syncthreads();
        u64 at = lower;
        for (int w = 0; w < warp; ++w) at += sh.warp_count[w];
        for (int i = i0; i < i1; i += 32) {
            const uint32_t set = __ballot_sync(0xffffffffu, tied(i + lane));
            const u64 place = at + __popc(set & ((2u << lane) - 1u));
            if (((set >> lane) & 1u) && place == need)
                for (int r = 0; r < C; ++r) st_remote32(remote(&sh.tie_limit, r), row.base + i + lane);
            at += __popc(set);
        }
    }
    cluster_sync();
    row.border = prefix;
    row.tie = sh.tie_limit;
    cluster_sync();
    return before + need * each;
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
    float x = DT == 0 ? static_cast<const float*>(p)[i]
                      : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    return x;
}
// NaN counts as -inf, -0 as +0.
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p) {
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared& sh = *reinterpret_cast<Shared*>(dyn);
    float* xs = reinterpret_cast<float*>(dyn + offset_slice(p.C));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank();
    const int C = p.C, m = blockIdx.x / C;
    pdl_wait();
    pdl_launch_dependents();

    Row row;
    row.base = (int)rank * p.slice;
    row.n = max(0, min(p.slice, p.V - row.base));
    row.x = xs;
    row.border = ~0ull;
    row.tie = 0xffffffffu;
    row.turn = 0;
    // the slice into shared memory; its largest logit, lowest index first
    const int64_t start = (int64_t)m * p.row_stride + row.base;
    u64 best = 0;
    auto see = [&](float x, int i) {
        xs[i] = x;
        const u64 k = ((u64)value_bits(x) << 32) | (uint32_t)~(uint32_t)(row.base + i);
        best = k > best ? k : best;
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
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
        best = other > best ? other : best;
    }
    if (lane == 0) sh.warp_mass[warp] = best;
    __syncthreads();
    if (tid < C) {
        for (int w = 0; w < kWarps; ++w) best = sh.warp_mass[w] > best ? sh.warp_mass[w] : best;
        st_remote64(remote(&sh.best[rank], tid), best);
    }
    cluster_sync();
    best = 0;
    for (int r = 0; r < C; ++r) best = sh.best[r] > best ? sh.best[r] : best;
    row.scale.top = bits_value((uint32_t)(best >> 32));
    const float T = p.temperature ? p.temperature[m] : 1.f;
    const int k = p.top_k ? p.top_k[m] : 0;
    const bool none = !(row.scale.top > -INFINITY);
    if (none || !(T > 0.f) || k == 1) {
        if (rank == 0 && tid == 0) {
            p.token[m] = none ? -1 : (int)~(uint32_t)best;
            if (p.prob) p.prob[m] = none ? 0.f : 1.f;
        }
        return;  // no CTA reads another's memory after the last barrier
    }
    const double c = fmin(1.4426950408889634 / (double)T, 1e30);
    row.scale.hi = (float)c;
    row.scale.lo = (float)(c - (double)row.scale.hi);

    const float top_p = p.top_p ? p.top_p[m] : 1.f;
    const bool by_p = top_p < 1.f;
    u64 total = 0;
    bool known = false;
    if (k > 0 && k < p.V) {
        total = narrow<false>(row, (u64)k, by_p, sh, rank, C);
        known = true;
    }
    if (by_p) {
        if (!known) {
            // the mass of everything
            u64 w = 0;
            for (int i = tid; i < row.n; i += kThreads) w += mass_of(xs[i], row.scale);
            w = warp_sum(w);
            if (lane == 0) sh.warp_mass[warp] = w;
            __syncthreads();
            row.turn ^= 1;
            if (tid < C) {
                u64 s = 0;
                for (int i = 0; i < kWarps; ++i) s += sh.warp_mass[i];
                st_remote64(remote(&sh.part_mass[row.turn][rank], tid), s);
            }
            cluster_sync();
            for (int r = 0; r < C; ++r) total += sh.part_mass[row.turn][r];
        }
        const double want = ceil((double)top_p * (double)total);
        narrow<true>(row, want >= 1.0 ? (u64)want : 1ull, true, sh, rank, C);
    }

    // the kept mass in index order: CTA by CTA, warp by warp
    const float min_p = p.min_p ? fminf(p.min_p[m], 1.f) : 0.f;
    const u64 least = min_p > 0.f ? (u64)ceil((double)min_p * (double)(1ull << kMassBits)) : 0ull;
    const uint32_t last_step = (uint32_t)(row.border >> 32);
    auto mass_at = [&](int i) -> u64 {
        const float x = xs[i];
        const uint32_t steps = steps_below(x, row.scale);
        if (steps > last_step || steps == 0xffffffffu) return 0;
        if (steps == last_step && !kept(row, code_of(steps, x), row.base + i)) return 0;
        const u64 w = mass_of(x, row.scale);
        return w >= least ? w : 0;
    };
    const int chunk = ((row.n + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int i0 = warp * chunk, i1 = min(i0 + chunk, row.n);
    u64 w = 0;
    for (int i = i0 + lane; i < i1; i += 32) w += mass_at(i);
    w = warp_sum(w);
    __syncthreads();
    if (lane == 0) sh.warp_mass[warp] = w;
    __syncthreads();
    row.turn ^= 1;
    if (tid < C) {
        u64 s = 0;
        for (int i = 0; i < kWarps; ++i) s += sh.warp_mass[i];
        st_remote64(remote(&sh.part_mass[row.turn][rank], tid), s);
    }
    cluster_sync();
    u64 before = 0, all = 0;
    for (int r = 0; r < C; ++r) {
        if (r < (int)rank) before += sh.part_mass[row.turn][r];
        all += sh.part_mass[row.turn][r];
    }
    for (int i = 0; i < warp; ++i) before += sh.warp_mass[i];
    const float u = p.u[m];
    u64 goal = u > 0.f ? (u64)((double)u * (double)all) : 0ull;
    if (!(u < 1.f) || goal >= all) goal = u > 0.f ? all - 1 : 0ull;
    if (before > goal || goal >= before + w) return;
    // this warp's chunk holds the token: the first with cdf > goal
    for (int i = i0; i < i1; i += 32) {
        const u64 own = i + lane < i1 ? mass_at(i + lane) : 0ull;
        u64 sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (before + sum - own <= goal && goal < before + sum) {
            p.token[m] = row.base + i + lane;
            if (p.prob) p.prob[m] = (float)((double)own / (double)all);
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        if (before > goal) break;
    }
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, int M, int dtype, cudaStream_t stream) {
    void (*kern)(SampleParams) = dtype == 0 ? sample_kernel<0> : sample_kernel<1>;
    const int smem = offset_slice(p.C) + p.slice * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && p.C > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(M * p.C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace moe
