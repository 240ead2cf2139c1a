// selective.h -- what the passes of the selective state-space scan share (selective.hip, selective_bwd.hip).
//
// A wavefront carries the states of 64 channels (one a lane in what a channel has once a token) by 16 states
// n. The tile lies in the registers as v_mfma_f32_16x16x1 (4 blocks) gives it: h[4 blk + r] of lane 16 q + j is
// state 4 q + r of channel 16 blk + j. That instruction adds a token's u (x) B to the decayed tile, from B_n
// in lane j = n and u in the channels' own lanes, in fp32 and beside the vector units, which bound these
// kernels: a state costs a product and an exponential (together three issue slots) for the decay, one product to
// apply it and one for y; what a channel has once a token costs a sixteenth of that. The steps reach the lanes of their
// channels' states through LDS (by permutes: 7% more time). Sums over n are over r in a lane and over q by two permlane
// swaps, which put channel c's sum in lane c.
#pragma once
#include <cmath>

#include "sdm_buffer.h"
#include "sdm_internal.h"
#include "sdm_rows.h"

// v_mul_legacy_f32: a product that is 0 where either factor is, whatever the other one is
extern "C" __device__ float sdm_mul_zero(float, float) __asm("llvm.amdgcn.fmul.legacy");

namespace sdm {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int SC = 8;               // tokens per chunk
constexpr float GONE = -INFINITY;   // in place of a sum of steps: a sequence began since, nothing crosses

template <bool BF16>
__device__ __forceinline__ float value(uint32_t u) {
    return BF16 ? bf16_f(u) : __uint_as_float(u);
}
// the address of element e (the same for the wavefront)
template <bool BF16>
__device__ __forceinline__ const char* row(const void* p, int64_t e) {
    return static_cast<const char*>(p) + e * (BF16 ? 2 : 4);
}

// Rows of tokens from token t on: a lane's element at vo bytes (OOB: nothing is read or written) of row i, with the
// row's offset in a scalar register. Token strides are below 2^26 elements, so that a chunk's rows lie within 2^31 bytes.
template <bool BF16>
struct Rows {
    rsrc_t r;
    uint32_t step;
    __device__ __forceinline__ Rows(const char* p, int64_t stride, int64_t t)
        : r(make_rsrc(row<BF16>(p, t * stride), 0x7FFFFFFF)), step((uint32_t)stride * (BF16 ? 2u : 4u)) {}
    __device__ __forceinline__ uint32_t get(uint32_t vo, uint32_t i) const {
        if constexpr (BF16) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)vo, (int)(i * step), 0);
        else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)vo, (int)(i * step), 0);
    }
    __device__ __forceinline__ void put(uint32_t vo, uint32_t i, float f) const {
        if constexpr (BF16) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f_bf16(f), r, (int)vo, (int)(i * step), 0);
        else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f), r, (int)vo, (int)(i * step), 0);
    }
};

// log(1 + e^v) = max(v, 0) + log(1 + e^-|v|); the logarithm of 1 + e as 2 artanh(s), s = e / (2 + e) <= 1/3, by a
// polynomial in s^2 (fitted at Chebyshev points; 5e-9 off at most, 8e-9 of the value): no worse for tiny e, where 1 + e in
// fp32 has lost it. e itself is off by its rounded argument, 1.25 |v| half steps of 2^-24 (|v| = 80: 4e-6 of a step of 2e-35).
__device__ __forceinline__ float softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(v));
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), w = s * s;
    float p = fmaf(0.28174657f, w, 0.27961418f);
    p = fmaf(p, w, 0.40024853f);
    p = fmaf(p, w, 0.66666317f);
    p = fmaf(p, w, 2.f);
    return fmaf(s, p, fmaxf(v, 0.f));
}

// The step: softplus(v), or v as it is. (A branch on it, which the compiler makes of a plain choice, would cut the token's
// instructions in pieces that are scheduled by themselves.)
__device__ __forceinline__ float step_of(float v, bool plus) {
    float s = softplus(v);
    asm volatile("" : "+v"(s));
    return plus ? s : v;
}

// v's four rows of 16 lanes, each in all rows
__device__ __forceinline__ void spread(float v, float (&o)[4]) {
    const uint32_t u = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    o[0] = __uint_as_float(a[0]); o[1] = __uint_as_float(a[1]);
    o[2] = __uint_as_float(b[0]); o[3] = __uint_as_float(b[1]);
}
// lane 16 blk + j: the sum of p[blk] over the lanes j, 16 + j, 32 + j, 48 + j
__device__ __forceinline__ float gather_sum(const float (&p)[4]) {
    auto add = [](auto h) { return __uint_as_float(h[0]) + __uint_as_float(h[1]); };
    const float s02 = add(__builtin_amdgcn_permlane32_swap(__float_as_uint(p[0]), __float_as_uint(p[2]), false, false));
    const float s13 = add(__builtin_amdgcn_permlane32_swap(__float_as_uint(p[1]), __float_as_uint(p[3]), false, false));
    return add(__builtin_amdgcn_permlane16_swap(__float_as_uint(s02), __float_as_uint(s13), false, false));
}

__device__ __forceinline__ f32x16 outer_add(float n, float c, f32x16 t) {
    return __builtin_amdgcn_mfma_f32_16x16x1f32(n, c, t, 0, 0, 0);
}

// Where a wavefront works
struct SelAt {
    int lane, q, j, nt;          // nt: tile of 16 states
    int64_t b, tile;             // tile: of channels, over all sequences and groups
    int g, c0, dg, seg;          // c0: first channel in its group
    bool in;                     // the lane's channel is there
    uint32_t c;                  // the lane's channel (the group's last one where it is not)
    uint32_t vo, vput;           // its offset in a row, in bytes; the same for stores, none where it is not there
    int64_t t0, t1, end;         // tokens of the segment, and those of them that are there
};
template <bool BF16, typename Args>
__device__ __forceinline__ SelAt sel_at(const Args& a) {
    SelAt w;
    w.lane = threadIdx.x & 63;
    w.q = w.lane >> 4;
    w.j = w.lane & 15;
    w.nt = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    w.tile = blockIdx.x;
    uint32_t i = blockIdx.x;
    w.c0 = (int)(i % (uint32_t)a.ctiles) * 64;
    i /= (uint32_t)a.ctiles;
    w.g = (int)(i % (uint32_t)a.G);
    w.b = i / (uint32_t)a.G;
    w.dg = a.D / a.G;
    w.in = w.c0 + w.lane < w.dg;
    w.c = (uint32_t)(w.g * w.dg + (w.in ? w.c0 + w.lane : w.dg - 1));
    w.vo = w.c * (BF16 ? 2u : 4u);
    w.vput = w.in ? w.vo : OOB;
    w.seg = blockIdx.y;
    w.t0 = (int64_t)w.seg * a.L;
    w.t1 = w.t0 + a.L < a.T ? w.t0 + a.L : a.T;
    int64_t n = a.T;
    if (a.lengths) {
        n = a.lengths[w.b];
        n = n < 0 ? 0 : n > a.T ? a.T : n;
    }
    w.end = n < w.t1 ? n : w.t1;
    return w;
}

// A tile out of [D][N] (of sequence b where there are several), zeros outside, times f
template <typename Args>
__device__ __forceinline__ f32x16 load_dn(const Args& a, const SelAt& w, const float* p, float f) {
    f32x16 v;
    const int n = 16 * w.nt + 4 * w.q;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = w.c0 + 16 * k + w.j;
        const float* e = p + (int64_t)(w.g * w.dg + c) * a.N + n;
        if (a.N % 4 == 0) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < w.dg && n < a.N) x = *reinterpret_cast<const float4*>(e);
            v[4 * k] = x.x * f; v[4 * k + 1] = x.y * f; v[4 * k + 2] = x.z * f; v[4 * k + 3] = x.w * f;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * k + r] = c < w.dg && n + r < a.N ? e[r] * f : 0.f;
        }
    }
    return v;
}
template <typename Args>
__device__ __forceinline__ void store_dn(const Args& a, const SelAt& w, float* p, const f32x16& v) {
    const int n = 16 * w.nt + 4 * w.q;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = w.c0 + 16 * k + w.j;
        if (c >= w.dg) continue;
        float* e = p + (int64_t)(w.g * w.dg + c) * a.N + n;
        if (a.N % 4 == 0) {
            if (n < a.N) *reinterpret_cast<float4*>(e) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N) e[r] = v[4 * k + r];
        }
    }
}

// Tiles in the workspace: 1024 floats as the registers hold them
__device__ __forceinline__ f32x16 load_tile(const float* p, int lane) {
    f32x16 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 x = reinterpret_cast<const float4*>(p)[64 * k + lane];
        v[4 * k] = x.x; v[4 * k + 1] = x.y; v[4 * k + 2] = x.z; v[4 * k + 3] = x.w;
    }
    return v;
}
__device__ __forceinline__ void store_tile(float* p, int lane, const f32x16& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        reinterpret_cast<float4*>(p)[64 * k + lane] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}

// exp(delta A) of the lane's 4 channels: a2 = A log2(e). At a sequence's first token delta is 0 and `gone` minus
// infinity (else 0): the decay is 0.
__device__ __forceinline__ f32x16 decays(const float4& delta, const f32x16& a2, float gone) {
    const float d[4] = {delta.x, delta.y, delta.z, delta.w};
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __builtin_amdgcn_exp2f(fmaf(d[i / 4], a2[i], gone));
    return v;
}
// d h, and 0 for a decay of 0 whatever h is: what a sequence left behind, a NaN among it, ends with it
__device__ __forceinline__ void decay(f32x16& h, const f32x16& d) {
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = sdm_mul_zero(d[i], h[i]);
}
__device__ __forceinline__ f32x16 zeros16() {
    f32x16 v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    return v;
}

// Bit k: a sequence begins at token t + k (k < 8, t + k < end)
__device__ __forceinline__ uint32_t starts(const uint8_t* start, int64_t t, int64_t end, int lane) {
    if (!start) return 0u;
    const bool on = lane < SC && t + lane < end && start[t + lane] != 0;
    return (uint32_t)__ballot(on);
}

// Values of B or C: lane 16 q + j gets state j's of token 4 k + q of a chunk (0 past its `left` tokens or the last state)
template <bool BF16>
__device__ __forceinline__ float load_bc(const Rows<BF16>& p, const SelAt& w, int k, int64_t left, int N) {
    const int n = 16 * w.nt + w.j, q = 4 * k + w.q;
    const uint32_t vo = q < left && n < N ? (uint32_t)q * p.step + (uint32_t)n * (BF16 ? 2u : 4u) : OOB;
    return value<BF16>(p.get(vo, 0));
}
// Row i of a chunk, or the last one that is there
__device__ __forceinline__ uint32_t upto(int i, int64_t left) { return i < left ? (uint32_t)i : (uint32_t)left - 1; }

// Tiles' ends carried through the segments: ends[s] holds what a segment adds (start state 0) and gets what
// arrives at it. A state a thread, the loads of 32 segments in flight together: their latency is what it takes
// (64 segments of 128 tiles: 19 us by 8 segments and 16 bytes a thread).
__global__ __launch_bounds__(256) void sel_carry_kernel(SelCarryArgs a0, SelCarryArgs a1) {
    const SelCarryArgs a = blockIdx.y ? a1 : a0;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // [tile][nt][blk][lane][r]
    const int e = (int)(i & 1023), r = e & 3, lane = e >> 2 & 63, blk = e >> 8, j = lane & 15, q = lane >> 4;
    const int64_t w = i >> 10, tile = w / a.ntiles;
    if (tile >= a.tiles) return;
    const int nt = (int)(w % a.ntiles);
    const int64_t bg = tile / a.ctiles, b = bg / a.G;
    const int g = (int)(bg % a.G), dg = a.D / a.G, c = (int)(tile % a.ctiles) * 64 + 16 * blk + j, n = 16 * nt + 4 * q + r;
    const bool in = c < dg && n < a.N;
    const int64_t at = ((int64_t)g * dg + c) * a.N + n;
    const float a2 = in ? a.A[at] * 1.44269504f : 0.f;
    float run = in && a.from ? a.from[b * a.D * a.N + at] : 0.f;
    const int64_t step = a.rev ? -1 : 1, first = a.rev ? a.nseg - 1 : 0;
    float* ends = a.ends + (first * a.tiles * a.ntiles + w) * 1024 + e;
    const float* sums = a.steps + (first * a.tiles + tile) * 64 + 16 * blk + j;
    const int64_t de = step * a.tiles * a.ntiles * 1024, ds = step * a.tiles * 64;
    constexpr int AHEAD = 32;
    for (int k = 0; k < a.nseg; k += AHEAD) {
        float own[AHEAD], sum[AHEAD];
#pragma unroll
        for (int m = 0; m < AHEAD; ++m) {
            own[m] = sum[m] = 0.f;
            if (k + m < a.nseg) {
                own[m] = ends[m * de];
                sum[m] = sums[m * ds];
            }
        }
#pragma unroll
        for (int m = 0; m < AHEAD; ++m) {
            if (k + m >= a.nseg) break;
            ends[m * de] = run;
            run = sum[m] == GONE ? own[m] : fmaf(__builtin_amdgcn_exp2f(a2 * sum[m]), run, own[m]);
        }
        ends += AHEAD * de;
        sums += AHEAD * ds;
    }
}
// Segments so that `waves` wavefronts work, of whole chunks and at least 16 tokens; with few channels as long as evens out the
// chains of a pass (some 0.3 us a token) and of the carry (0.06 a segment): the root of T / 10 tokens (one sequence of
// 131072 x 64: 810 us by segments of 16, 215 of 120; 8192 x 64: 66 and 51 of 32; of T / 4: no faster, backwards up to 18% slower)
inline void sel_segments(int64_t B, int64_t T, int G, int D, int N, int64_t waves, int64_t* L, int* nseg) {
    const int64_t per = sel_tiles(B, G, D) * sel_ntiles(N), want = (waves + per - 1) / per;
    int64_t len = (T + want - 1) / want;
    const int64_t least = (int64_t)sqrt(0.1 * (double)T);
    if (len < least) len = least;
    if (len < 16) len = 16;
    len = (len + SC - 1) / SC * SC;
    *L = len;
    *nseg = T > len ? (int)((T + len - 1) / len) : 1;
}

inline hipError_t sel_carry(const SelCarryArgs& a, const SelCarryArgs& b, int count, hipStream_t st) {
    hipLaunchKernelGGL(sel_carry_kernel, dim3((unsigned)(a.tiles * a.ntiles * 4), count), dim3(256), 0, st, a, b);
    return hipGetLastError();
}

}  // namespace
}  // namespace sdm
