// selective.hip -- the selective state-space scan on gfx950: for every channel d and state n
//   delta_t = softplus(dt_t + bias),   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
//   y_t = (sum_n C_t h_t + D x_t) silu(z_t),
// for prompts, long sequences and single tokens (states in place), packed or padded.
//
// With few streams of channels the tokens are cut into segments: a first pass leaves what each adds to a state
// of zeros and its sum of steps (a segment's decay is exp(A times that)), a carry runs through them, and the
// last pass starts every segment where it belongs. See selective.h for a wavefront's tile.
//
// Bound by vector instructions (103 a token and tile in the last pass, 74 in the first; issued in 96% of the cycles):
// 4 x 8192 x 2048 with 16 states in bf16, 171 to 185 us first pass, 18 carry and 232 to 251 last pass (422 a call), for 105 us
// of HBM at a copy's rate and 137 of one pass's exponentials and products alone; one token of 256 sequences 15.3 us (71 MB,
// 4.7 TB/s): HBM.
#include <cmath>
#include <type_traits>

#include "selective.h"

namespace sdm {
namespace {

constexpr int SEL_SHARE = SC * 16 + SC * 16 / 4;  // LDS of a wavefront in 16 bytes: a chunk's steps and its C

// EMIT: the pass that writes y and the last state; else the first pass. MULTI: several tiles of states, one
// a wavefront, whose shares of y are added in their order. ONE: single tokens, in 60 registers in place of 116, so
// that twice the wavefronts have their states' loads in flight (256 sequences of 2048 x 16 17.3 -> 15.4 us, 512: 29.5 -> 25.4).
template <bool BF16, bool HASZ, bool MULTI, bool EMIT, bool ONE>
__global__ __launch_bounds__(MULTI ? 256 : 64, ONE ? 6 : 3) void sel_kernel(SelArgs a) {
    constexpr int TOK = ONE ? 1 : SC, QS = (TOK + 3) / 4;  // tokens at once, and their quarters of a wavefront
    extern __shared__ float4 lds4[];  // a wavefront's share, then the shares of y: [2][ntiles][SC][64]
    const SelAt w = sel_at<BF16>(a);
    float4(*dl)[16] = reinterpret_cast<float4(*)[16]>(lds4 + w.nt * SEL_SHARE);  // a chunk's steps: a lane's 4 channels side by side
    float(*cl)[16] = reinterpret_cast<float(*)[16]>(dl + SC);
    float(*yl)[SC][64] = reinterpret_cast<float(*)[SC][64]>(lds4 + a.ntiles * SEL_SHARE);
    const f32x16 a2 = load_dn(a, w, a.A, 1.44269504f);
    const int64_t wave = w.tile * a.ntiles + w.nt, waves = a.tiles * a.ntiles, per = (int64_t)a.D * a.N;
    f32x16 h = zeros16();
    if constexpr (EMIT) {
        if (a.nseg > 1) h = load_tile(a.ends + (w.seg * waves + wave) * 1024, w.lane);
        else if (a.S0) h = load_dn(a, w, a.S0 + w.b * per, 1.f);
    }
    const char* px = row<BF16>(a.x, w.b * a.x_b);
    const char* pd = row<BF16>(a.dt, w.b * a.dt_b);
    const char* pz = HASZ ? row<BF16>(a.z, w.b * a.z_b) : nullptr;
    const char* pB = row<BF16>(a.Bm, w.b * a.B_b + w.g * a.B_g);
    const char* pC = EMIT ? row<BF16>(a.Cm, w.b * a.C_b + w.g * a.C_g) : nullptr;
    const char* py = EMIT ? row<BF16>(a.y, w.b * a.T * a.D) : nullptr;
    const float bias = a.bias ? a.bias[w.c] : 0.f, skip = EMIT && a.Dskip ? a.Dskip[w.c] : 0.f;
    const uint8_t* start = a.start ? a.start + w.b * a.T : nullptr;
    float steps = 0.f;
    bool cut = false;  // a sequence began in the segment: nothing crosses it
    int par = 0;
    // A chunk's inputs: the first `left` of its tokens
    struct Chunk {
        uint32_t x[TOK], d[TOK], z[TOK];
        float b[QS], c[QS];
        uint32_t st;
    };
    auto fetch = [&](auto whole, int64_t t, int64_t left) {
        constexpr bool ALL = decltype(whole)::value;
        const Rows<BF16> X(px, a.x_t, t), T(pd, a.dt_t, t), Z(pz, HASZ ? a.z_t : 0, HASZ ? t : 0);
        const Rows<BF16> B(pB, a.B_t, t), C(pC, EMIT ? a.C_t : 0, EMIT ? t : 0);
        Chunk f;
#pragma unroll
        for (int i = 0; i < TOK; ++i)
            if (ALL || i < left) {
                f.x[i] = X.get(w.vo, i);
                f.d[i] = T.get(w.vo, i);
                if constexpr (HASZ && EMIT) f.z[i] = Z.get(w.vo, i);
            }
#pragma unroll
        for (int k = 0; k < QS; ++k) {
            f.b[k] = load_bc(B, w, k, left, a.N);
            if constexpr (EMIT) f.c[k] = load_bc(C, w, k, left, a.N);
        }
        f.st = starts(start, t, w.end, w.lane);
        return f;
    };
    // all 8 tokens of a chunk, or the `left` ones at the end (a branch for each: one token costs one)
    auto chunk = [&](auto whole, const Chunk& f, int64_t t, int64_t left) {
        constexpr bool ALL = decltype(whole)::value;
        const Rows<BF16> Y(py, EMIT ? a.D : 0, EMIT ? t : 0);
        if constexpr (!EMIT) cut |= f.st != 0;
        float bq[QS][4];
#pragma unroll
        for (int k = 0; k < QS; ++k) {
            spread(f.b[k], bq[k]);
            if constexpr (EMIT) cl[4 * k + w.q][w.j] = f.c[k];
        }
        float u[TOK];
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            if (!ALL && i >= left) break;
            const float delta = step_of(value<BF16>(f.d[i]) + bias, a.softplus);
            u[i] = delta * value<BF16>(f.x[i]);
            if constexpr (!EMIT) steps += delta;
            reinterpret_cast<float*>(dl[i])[4 * w.j + w.q] = f.st >> i & 1u ? 0.f : delta;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // y's last steps: D x and the gate (a lane without a channel works on the last one's rows, and stores nothing)
        auto finish = [&](int i, float y) {
            float o = fmaf(skip, value<BF16>(f.x[i]), y);
            if constexpr (HASZ) {
                const float z = value<BF16>(f.z[i]);
                o *= z * sigmoid(z);
            }
            Y.put(w.vput, i, o);
        };
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            if (!ALL && i >= left) break;
            decay(h, decays(dl[i][w.j], a2, f.st >> i & 1u ? GONE : 0.f));
            h = outer_add(bq[i / 4][i % 4], u[i], h);
            if constexpr (EMIT) {
                const float4 c = *reinterpret_cast<const float4*>(&cl[i][4 * w.q]);
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = fmaf(c.w, h[4 * k + 3], fmaf(c.z, h[4 * k + 2], fmaf(c.y, h[4 * k + 1], c.x * h[4 * k])));
                const float y = gather_sum(p);
                if constexpr (MULTI) yl[par * a.ntiles + w.nt][i][w.lane] = y;
                else finish(i, y);
            }
        }
        if constexpr (MULTI && EMIT) {
            __syncthreads();  // (the other half of yl: its readers have passed the barrier before)
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                if (i % a.ntiles != w.nt || (!ALL && i >= left)) continue;
                float y = 0.f;
                for (int k = 0; k < a.ntiles; ++k) y += yl[par * a.ntiles + k][i][w.lane];
                finish(i, y);
            }
            par ^= 1;
        }
    };
    int64_t t = w.t0;
    if constexpr (EMIT && !ONE) {
        for (; t + SC <= w.end; t += SC) chunk(std::true_type{}, fetch(std::true_type{}, t, SC), t, SC);
    } else if (!EMIT && t + SC <= w.end) {  // a chunk ahead (203 -> 195 us; with z it would take a wavefront's room a SIMD: 272 -> 276)
        Chunk f = fetch(std::true_type{}, t, SC);
        for (; t + 2 * SC <= w.end; t += SC) {
            const Chunk next = fetch(std::true_type{}, t + SC, SC);
            chunk(std::true_type{}, f, t, SC);
            f = next;
        }
        chunk(std::true_type{}, f, t, SC);
        t += SC;
    }
    if (t < w.end) chunk(std::false_type{}, fetch(std::false_type{}, t, w.end - t), t, w.end - t);
    if constexpr (EMIT) {
        if (w.nt == 0)
            for (int64_t t = w.end > w.t0 ? w.end : w.t0; t < w.t1; ++t) Rows<BF16>(py, a.D, t).put(w.vput, 0, 0.f);
        if (a.S && w.seg == a.nseg - 1) store_dn(a, w, a.S + w.b * per, h);
    } else {
        store_tile(a.ends + (w.seg * waves + wave) * 1024, w.lane, h);
        if (w.nt == 0) a.steps[(w.seg * a.tiles + w.tile) * 64 + w.lane] = cut ? GONE : steps;
    }
}

template <bool BF16, bool HASZ, bool EMIT, bool ONE>
void sel_go(const SelArgs& a, int nseg, hipStream_t st) {
    const dim3 grid((unsigned)a.tiles, (unsigned)nseg);
    const int lds = SEL_SHARE * 16 * a.ntiles;
    if (a.ntiles > 1) hipLaunchKernelGGL((sel_kernel<BF16, HASZ, true, EMIT, ONE>), grid, dim3(64 * a.ntiles), lds + (EMIT ? 2 * a.ntiles * SC * 256 : 0), st, a);
    else hipLaunchKernelGGL((sel_kernel<BF16, HASZ, false, EMIT, ONE>), grid, dim3(64), lds, st, a);
}
template <bool ONE>
void sel_emit(const SelArgs& a, hipStream_t st) {
    if (a.z) a.bf16 ? sel_go<true, true, true, ONE>(a, a.nseg, st) : sel_go<false, true, true, ONE>(a, a.nseg, st);
    else a.bf16 ? sel_go<true, false, true, ONE>(a, a.nseg, st) : sel_go<false, false, true, ONE>(a, a.nseg, st);
}

// One segment where that takes no longer, by estimates in microseconds. A token after the other: 0.32 of one wavefront a
// SIMD, 0.45 where every SIMD has one, 0.19 more for each further one, and 0.15 or 0.06 where wavefronts meet in a workgroup. Cut:
// two more launches, and both passes' vector instructions, 4.1e-4 a token and wavefront. (One segment / cut, 16 states, 2048
// channels; 1 sequence of 32 tokens: 15.7 / 19.2, of 64: 26 / 19.6; 8 of 64: 26.6 / 27.1; 32 of 160: 73 / 93, of 1024:
// 458 / 407; 48 of 1024: 561 / 597; 100 of 1024: 948 / 1171. Near the crossing the choice costs up to 6%.)
// Cut into 8192 wavefronts, twice what fits: shorter ones even out what padding leaves uneven (2 x 40001 x 520 with one
// sequence padded: 714 with 4096, 654 so).
void sel_split(int64_t B, int64_t T, int G, int D, int N, int64_t* L, int* nseg) {
    const double per = (double)(sel_tiles(B, G, D) * sel_ntiles(N)), full = per / 1024.0;
    const bool multi = sel_ntiles(N) > 1;
    const double token = full <= 1.0 ? 0.32 + 0.13 * full + (multi ? 0.15 : 0.0) : 0.18 + 0.19 * ceil(full) + (multi ? 0.06 : 0.0);
    const bool cut = 4.0 + token * (double)T > 18.0 + 6.0 * full + 4.1e-4 * per * (double)T;
    sel_segments(B, T, G, D, N, cut ? 8192 : 1, L, nseg);
}

}  // namespace

int64_t selective_workspace_bytes(int64_t B, int64_t T, int G, int D, int N) {
    int64_t L;
    int nseg;
    sel_split(B, T, G, D, N, &L, &nseg);
    return nseg > 1 ? nseg * sel_tiles(B, G, D) * (sel_ntiles(N) * 4096 + 256) : 0;
}

hipError_t launch_selective(SelArgs a, hipStream_t st) {
    a.ctiles = sel_ctiles(a.G, a.D);
    a.ntiles = sel_ntiles(a.N);
    a.tiles = sel_tiles(a.B, a.G, a.D);
    sel_split(a.B, a.T, a.G, a.D, a.N, &a.L, &a.nseg);
    a.ends = static_cast<float*>(a.workspace);
    a.steps = a.ends + a.nseg * a.tiles * a.ntiles * 1024;
    if (a.nseg > 1) {
        a.bf16 ? sel_go<true, false, false, false>(a, a.nseg - 1, st) : sel_go<false, false, false, false>(a, a.nseg - 1, st);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        SelCarryArgs c{};
        c.ends = a.ends; c.steps = a.steps; c.A = a.A; c.from = a.S0;
        c.tiles = a.tiles; c.nseg = a.nseg; c.ntiles = a.ntiles; c.ctiles = a.ctiles; c.G = a.G; c.D = a.D; c.N = a.N;
        if ((e = sel_carry(c, c, 1, st)) != hipSuccess) return e;
    }
    a.T == 1 ? sel_emit<true>(a, st) : sel_emit<false>(a, st);
    return hipGetLastError();
}

}  // namespace sdm
