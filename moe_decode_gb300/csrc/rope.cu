// Rotary positions (moe_rope), alone or in one pass with the write of keys and
// values into a paged cache of 16-bit values or of e4m3 codes, and the reading
// back of slots (moe_paged_rope_append and its kin, moe_paged_read).
#include <algorithm>

#include "layer_params.h"
#include "paged.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPitch = 33;  // an eighth of the pairs of a head of 512 dimensions, and one
// Rounds whose loads are on their way together, and CTAs of an SM: 8,192 tokens of
// 32 and 8 heads of 128 take 34.8 us with (4, 2), 32.2 with (2, 3), 28.2 with (2, 4).
constexpr int kRounds = 2, kCtas = 4;

__device__ __forceinline__ void report_slot(unsigned* ctrl) {
    atomicCAS(reinterpret_cast<int*>(ctrl + kCtlStatus), 0, -100 /* MOE_EDEVICE_BAD_INDEX */);
}

template <int DT>
__device__ __forceinline__ float2 widen(uint32_t v) {
    return DT == 0 ? make_float2(bf16lo(v), bf16hi(v)) : f16x2_to_f32(v);
}
template <int DT>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
    uint32_t d;
    if (DT == 0) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// cos and sin of a fraction of a turn in 2^-32: the nearest quarter by integers,
// so that the rest, at most an eighth of a turn, loses nothing in fp32.
__device__ __forceinline__ float2 turn(uint32_t phase) {
    const uint32_t quarter = (phase + (1u << 29)) >> 30;
    const int rest = (int)(phase - (quarter << 30));
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    const float x = quarter & 1u ? -s : c, y = quarter & 1u ? c : s;
    return quarter & 2u ? make_float2(-x, -y) : make_float2(x, y);
}

// (a, b) turned by (c, s), pairs of 16-bit values.
template <int DT>
__device__ __forceinline__ void turn2(uint32_t& a, uint32_t& b, const float2 (&cs)[2]) {
    const float2 x = widen<DT>(a), y = widen<DT>(b);
    a = narrow<DT>(x.x * cs[0].x - y.x * cs[0].y, x.y * cs[1].x - y.y * cs[1].y);
    b = narrow<DT>(x.x * cs[0].y + y.x * cs[0].x, x.y * cs[1].y + y.y * cs[1].x);
}

// Four values into four e4m3 codes, in order from the low byte.
__device__ __forceinline__ uint32_t codes4(float2 a, float2 b) {
    uint32_t d;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(d)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A token's heads (queries, keys, values in that order) go to `split` warps, in
// rounds of p.per heads: a lane has 16 of a head's elements, as two pieces of 8
// that are each other's partners where pairs lie half the rotated part apart.
// The token's cosines and sines are computed once a warp and read by all its
// rounds. With a cache of codes the head's lanes find its largest magnitude by
// shuffles.
template <int DT, int TO>
__global__ __launch_bounds__(kThreads, kCtas) void rotate_kernel(const __grid_constant__ RotateParams p) {
    // pair 8 i + j at j * kPitch + i: lanes of a head read neighbours
    __shared__ float2 table[kWarps][8 * kPitch];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane / p.lanes, i = lane - sub * p.lanes;
    const bool turns = p.positions != nullptr && 16 * i < p.rotary_dim;
    // the two pieces: partners, or neighbours
    int at0 = 16 * i, at1 = 16 * i + 8;
    if (p.positions != nullptr && !p.interleaved && turns) {
        at0 = 8 * i;
        at1 = 8 * i + p.rotary_dim / 2;
    }
    const int heads = p.heads[0] + p.heads[1] + p.heads[2];
    const int rounds = (heads + p.per - 1) / p.per;
    const int64_t all = (int64_t)p.T * p.split, step = (int64_t)gridDim.x * kWarps;
    for (int64_t w = (int64_t)blockIdx.x * kWarps + warp; w < all; w += step) {
        const int t = (int)(w / p.split), part = (int)(w - (int64_t)t * p.split);
        const int pos = p.positions ? p.positions[t] : 0;
        int slot = TO != kRotateRows ? p.slots[t] : -1;
        if (pos < 0) continue;
        if (TO != kRotateRows && (slot < -1 || slot >= p.n_slots)) {
            if (lane == 0 && part == 0) report_slot(p.ctrl);
            slot = -1;
        }
        const int block = slot < 0 ? 0 : slot / p.block_size, token = slot < 0 ? 0 : slot - block * p.block_size;
        uint8_t* to[2] = {};
        if (TO != kRotateRows)
#pragma unroll
            for (int n = 0; n < 2; ++n) to[n] = p.cache[n] + block * p.cache_block[n] + token * p.cache_token[n];
        // `kRounds` rounds from r0 on: which head this lane has of each (kind 0
        // queries, 1 keys, 2 values, -1 nothing), and its pieces on their way
        uint4 a[kRounds], b[kRounds];
        int kind[kRounds], head[kRounds];
        const uint16_t* const from[3] = {p.src[0] + t * p.src_token[0], p.src[1] + t * p.src_token[1], p.src[2] + t * p.src_token[2]};
        auto load = [&](int r0) {
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                const int r = r0 + u * p.split;
                int h = r * p.per + sub;
                kind[u] = -1;
                if (r < rounds && sub < p.per && h < heads) {
                    kind[u] = 0;
                    if (h >= p.heads[0]) {
                        h -= p.heads[0];
                        kind[u] = 1;
                        if (h >= p.heads[1]) {
                            h -= p.heads[1];
                            kind[u] = 2;
                        }
                    }
                    if (TO != kRotateRows && slot < 0 && kind[u] > 0) kind[u] = -1;
                }
                head[u] = h;
                a[u] = b[u] = make_uint4(0, 0, 0, 0);
                if (kind[u] >= 0) {
                    const int k = kind[u];
                    const uint16_t* s = (k == 0 ? from[0] : k == 1 ? from[1] : from[2]) +
                                        h * (k == 0 ? p.src_head[0] : k == 1 ? p.src_head[1] : p.src_head[2]);
                    a[u] = *reinterpret_cast<const uint4*>(s + at0);
                    b[u] = *reinterpret_cast<const uint4*>(s + at1);
                }
            }
        };
        load(part);
        float2 cs[8];
        if (p.positions) {
            __syncwarp();
            for (int j = lane; j < p.rotary_dim / 2; j += 32) {
                const float2 c = turn((uint32_t)(((unsigned long long)(unsigned)pos * __ldg(p.turns + j)) >> 32));
                table[warp][(j & 7) * kPitch + (j >> 3)] = make_float2(c.x * p.scale, c.y * p.scale);
            }
            __syncwarp();
            if (turns)
#pragma unroll
                for (int j = 0; j < 8; ++j) cs[j] = table[warp][j * kPitch + i];
        }
        for (int r0 = part; r0 < rounds; r0 += kRounds * p.split) {
            if (r0 != part) load(r0);
#pragma unroll
            for (int u = 0; u < kRounds; ++u) {
                const int k = kind[u];
                uint32_t* x = reinterpret_cast<uint32_t*>(&a[u]);
                uint32_t* y = reinterpret_cast<uint32_t*>(&b[u]);
                if (turns && (k == 0 || k == 1)) {
                    if (p.interleaved) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            uint32_t& z = j < 4 ? x[j & 3] : y[j & 3];
                            const float2 v = widen<DT>(z);
                            z = narrow<DT>(v.x * cs[j].x - v.y * cs[j].y, v.x * cs[j].y + v.y * cs[j].x);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 c[2] = {cs[2 * j], cs[2 * j + 1]};
                            turn2<DT>(x[j], y[j], c);
                        }
                    }
                }
                if (TO == kRotateRows || k == 0) {
                    if (k < 0) continue;
                    uint16_t* d = (k == 0 ? p.dst[0] : p.dst[1]) + t * (k == 0 ? p.dst_token[0] : p.dst_token[1]) +
                                  head[u] * (k == 0 ? p.dst_head[0] : p.dst_head[1]);
                    *reinterpret_cast<uint4*>(d + at0) = a[u];
                    *reinterpret_cast<uint4*>(d + at1) = b[u];
                    if (TO != kRotateCache8) continue;
                }
                const int n = k == 2 ? 1 : 0;  // keys, values
                if (TO == kRotateCache16 && k > 0) {
                    uint8_t* row = to[n] + head[u] * p.cache_head[n];
                    *reinterpret_cast<uint4*>(row + 2 * at0) = a[u];
                    *reinterpret_cast<uint4*>(row + 2 * at1) = b[u];
                }
                if (TO == kRotateCache8 && __any_sync(0xffffffffu, k > 0)) {
                    // the largest magnitude of the head, of bits without their
                    // signs, in which NaN comes above infinity above all others
                    uint32_t most = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) most = __vmaxu2(most, __vmaxu2(x[j] & 0x7fff7fffu, y[j] & 0x7fff7fffu));
                    most = max(most & 0xffffu, most >> 16);
                    for (int o = 1; o < p.lanes; o <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
                    const uint32_t top = __float_as_uint(widen<DT>(most).x);
                    // 240 of the largest power of two: what lies above it is rounded
                    // down to it, as 256 of them is the first value beyond the type
                    constexpr uint32_t kLast = DT == 0 ? 0x7f70u : 0x7b80u;
                    if (most > kLast) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[j] = (x[j] & 0x80008000u) | __vminu2(x[j] & 0x7fff7fffu, kLast * 0x10001u);
                            y[j] = (y[j] & 0x80008000u) | __vminu2(y[j] & 0x7fff7fffu, kLast * 0x10001u);
                        }
                    }
                    if (k > 0) {
                        // 448 is 1.75 * 2^8
                        int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
                        e = max(e, -127);
                        const bool finite = top < 0x7f800000u;
                        const float by = finite ? exp2i(-e) : 0.f;
                        uint32_t c[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                        {
                            const float2 f = widen<DT>(j < 2 ? x[2 * j & 3] : y[2 * j & 3]), g = widen<DT>(j < 2 ? x[(2 * j + 1) & 3] : y[(2 * j + 1) & 3]);
                            c[j] = finite ? codes4(make_float2(f.x * by, f.y * by), make_float2(g.x * by, g.y * by)) : 0u;
                        }
                        uint8_t* row = to[n] + head[u] * p.cache_head[n];
                        *reinterpret_cast<uint2*>(row + at0) = make_uint2(c[0], c[1]);
                        *reinterpret_cast<uint2*>(row + at1) = make_uint2(c[2], c[3]);
                        if (i == 0)
                            p.cache_scale[n][((int64_t)block * p.heads[1] + head[u]) * p.block_size + token] =
                                (uint8_t)(finite ? e + 127 : 255);
                    }
                }
            }
        }
    }
}

// A token's heads of keys, then of values, to `split` warps; a lane has 16
// elements of a head, four of them on their way at a time.
template <int FROM, int DT>
__global__ __launch_bounds__(kThreads) void read_kernel(const __grid_constant__ ReadParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int units = p.heads << p.lane_shift, mask = (1 << p.lane_shift) - 1;
    const int64_t all = (int64_t)p.T * p.split, step = (int64_t)gridDim.x * kWarps;
    for (int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); w < all; w += step) {
        const int t = (int)(w / p.split), part = (int)(w - (int64_t)t * p.split);
        const int slot = p.slots[t];
        if (slot < 0 || slot >= p.n_slots) {
            if (slot != -1 && lane == 0 && part == 0) report_slot(p.ctrl);
            continue;
        }
        const int block = slot / p.block_size, token = slot - block * p.block_size;
        constexpr int U = 4;
        for (int c0 = part * 32 + lane; c0 < 2 * units; c0 += U * 32 * p.split) {
            uint4 v[U], v2[U];
            uint32_t scale[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * 32 * p.split;
                if (c < 2 * units) {
                    const int n = c >= units, x = c - n * units, head = x >> p.lane_shift, i = x & mask;
                    const uint8_t* row = p.cache[n] + block * p.cache_block[n] + token * p.cache_token[n] + head * p.cache_head[n];
                    if (FROM == 1) {
                        v[u] = *reinterpret_cast<const uint4*>(row + 16 * i);
                        scale[u] = p.cache_scale[n][((int64_t)block * p.heads + head) * p.block_size + token];
                    } else {
                        v[u] = *reinterpret_cast<const uint4*>(row + 32 * i);
                        v2[u] = *reinterpret_cast<const uint4*>(row + 32 * i + 16);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * 32 * p.split;
                if (c >= 2 * units) break;
                const int n = c >= units, x = c - n * units, head = x >> p.lane_shift, i = x & mask;
                uint16_t* d = p.dst[n] + t * p.dst_token[n] + head * p.dst_head[n] + 16 * i;
                if (FROM == 1) {
                    float2 f[8];
                    unpack16_e4m3x2(v[u], f);
                    const float by = e8m0_to_f32(scale[u]);
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = narrow<DT>(f[j].x * by, f[j].y * by);
                    *reinterpret_cast<uint4*>(d) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(d + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                } else {
                    *reinterpret_cast<uint4*>(d) = v[u];
                    *reinterpret_cast<uint4*>(d + 8) = v2[u];
                }
            }
        }
    }
}

template <class P>
cudaError_t launch_pdl(void (*kern)(P), int grid, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// The warps that share a token: `warps` of an SM are wanted, each with a round at
// the least.
int split_of(int T, int rounds, int sms, int warps) {
    const int64_t want = ((int64_t)sms * warps + T - 1) / T;
    return (int)(want > rounds ? rounds : want);
}
int grid_of(int64_t warps, int64_t most) {
    const int64_t want = (warps + kWarps - 1) / kWarps;
    return (int)(want > most ? most : want);
}

}  // namespace

cudaError_t launch_rotate(RotateParams p, int to, int dtype, int sms, cudaStream_t stream) {
    p.lanes = p.head_dim / 16;
    p.per = 32 / p.lanes;
    const int heads = p.heads[0] + p.heads[1] + p.heads[2], rounds = (heads + p.per - 1) / p.per;
    // Each warp of a token computes the token's angles. Enough of them to have 16 an
    // SM, and while there are tokens for fewer than 160, as many as leave each four
    // rounds. (us by 16, by 160, by this: 32/8 heads of 128 into codes, 1,024 tokens
    // 8.9, 11.6, 8.9, 2,048 14.5, 20.3, 16.5, 4,096 24.3, 24.7, 23.8, 8,192 42.2, 39.7,
    // 39.7, 20,000 91.7, 85.0, 84.9; 8/2 heads, 8,192 tokens 16.0, 20.6, 16.1; 64/8
    // heads, 1,024 tokens 14.4, 17.5, 14.7, 8,192 65.8, 61.8, 61.8.)
    p.split = std::max(split_of(p.T, rounds, sms, 16), std::min(split_of(p.T, rounds, sms, 160), (rounds + 3) / 4));
    const int grid = grid_of((int64_t)p.T * p.split, (int64_t)sms * 8);
    if (dtype == 0) {
        if (to == kRotateRows) return launch_pdl(rotate_kernel<0, kRotateRows>, grid, p, stream);
        if (to == kRotateCache16) return launch_pdl(rotate_kernel<0, kRotateCache16>, grid, p, stream);
        return launch_pdl(rotate_kernel<0, kRotateCache8>, grid, p, stream);
    }
    if (to == kRotateRows) return launch_pdl(rotate_kernel<1, kRotateRows>, grid, p, stream);
    if (to == kRotateCache16) return launch_pdl(rotate_kernel<1, kRotateCache16>, grid, p, stream);
    return launch_pdl(rotate_kernel<1, kRotateCache8>, grid, p, stream);
}

cudaError_t launch_read(ReadParams p, int from, int dtype, int sms, cudaStream_t stream) {
    const int rounds = ((2 * p.heads << p.lane_shift) + 31) / 32;
    p.split = split_of(p.T, rounds, sms, 64);
    // (CTAs without a second token: 65,521 tokens 63.5 us, 69.3 by 8 an SM in turn)
    const int grid = grid_of((int64_t)p.T * p.split, (int64_t)sms * 64);
    if (from == 0) return launch_pdl(read_kernel<0, 0>, grid, p, stream);
    return dtype == 0 ? launch_pdl(read_kernel<1, 0>, grid, p, stream) : launch_pdl(read_kernel<1, 1>, grid, p, stream);
}

}  // namespace moe
