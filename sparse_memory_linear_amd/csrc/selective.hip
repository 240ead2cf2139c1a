// selective.hip -- the selective state-space scan on gfx950: for every channel d and state n
//   delta_t = softplus(dt_t + bias),   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
//   y_t = (sum_n C_t h_t + D x_t) silu(z_t),
// for prompts, long sequences and single tokens (states in place), packed or padded.
//
// With few streams of channels the tokens are cut into segments: a first pass leaves what each adds to a state
// of zeros and its sum of steps (a segment's decay is exp(A times that)), a carry runs through them, and the
// last pass starts every segment where it belongs. See selective.h for a wavefront's tile.
#include "selective.h"

namespace sdm {
namespace {

// EMIT: the pass that writes y and the last state; else the first pass. MULTI: several tiles of states, one
// a wavefront, whose shares of y are added in their order.
template <bool BF16, bool HASZ, bool MULTI, bool EMIT>
__global__ __launch_bounds__(MULTI ? 256 : 64, 3) void sel_kernel(SelArgs a) {
    constexpr int NW = MULTI ? 4 : 1;
    __shared__ float cl[NW][SC][16];
    __shared__ float yl[MULTI && EMIT ? 2 : 1][NW][MULTI && EMIT ? SC : 1][64];
    const SelAt w = sel_at(a);
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
    const float bias = a.bias ? a.bias[w.c] : 0.f, skip = EMIT && a.Dskip ? a.Dskip[w.c] : 0.f;
    const uint8_t* start = a.start ? a.start + w.b * a.T : nullptr;
    float steps = 0.f;
    int par = 0;
    for (int64_t t = w.t0; t < w.end; t += SC) {
        uint32_t xr[SC], dr[SC], zr[SC];
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const int64_t u = t + i < w.end ? t + i : w.end - 1;
            xr[i] = raw<BF16>(row<BF16>(px, u * a.x_t), w.c);
            dr[i] = raw<BF16>(row<BF16>(pd, u * a.dt_t), w.c);
            if constexpr (HASZ && EMIT) zr[i] = raw<BF16>(row<BF16>(pz, u * a.z_t), w.c);
        }
        const float b0 = load_bc<BF16>(pB, a.B_t, t, w, a.N), b1 = load_bc<BF16>(pB, a.B_t, t + 4, w, a.N);
        if constexpr (EMIT) {
            const float c0 = load_bc<BF16>(pC, a.C_t, t, w, a.N), c1 = load_bc<BF16>(pC, a.C_t, t + 4, w, a.N);
            cl[w.nt][w.q][w.j] = c0;
            cl[w.nt][4 + w.q][w.j] = c1;
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        const uint32_t st = starts(start, t, w.end, w.lane);
        float bq[2][4];
        spread(b0, bq[0]);
        spread(b1, bq[1]);
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const bool on = w.in && t + i < w.end;
            const float v = value<BF16>(dr[i]) + bias, x = value<BF16>(xr[i]);
            float delta = a.softplus ? softplus(v) : v;
            delta = on ? delta : 0.f;
            const float u = on ? delta * x : 0.f;
            if constexpr (!EMIT) steps = st >> i & 1u ? GONE : steps + delta;
            if (st >> i & 1u) {
                h = zeros16();
            } else {
                const f32x16 d = decays(delta, a2);
#pragma unroll
                for (int k = 0; k < 16; ++k) h[k] *= d[k];
            }
            h = outer_add(bq[i / 4][i % 4], u, h);
            if constexpr (EMIT) {
                const float4 c = *reinterpret_cast<const float4*>(&cl[w.nt][i][4 * w.q]);
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    p[k] = fmaf(c.w, h[4 * k + 3], fmaf(c.z, h[4 * k + 2], fmaf(c.y, h[4 * k + 1], c.x * h[4 * k])));
                const float y = gather_sum(p);
                if constexpr (MULTI) {
                    yl[par][w.nt][i][w.lane] = y;
                } else if (on) {
                    float o = fmaf(skip, x, y);
                    if constexpr (HASZ) {
                        const float z = value<BF16>(zr[i]);
                        o *= z * sigmoid(z);
                    }
                    put<BF16>(const_cast<char*>(row<BF16>(a.y, (w.b * a.T + t + i) * a.D)), w.c, o);
                }
            }
        }
        if constexpr (MULTI && EMIT) {
            __syncthreads();  // the other half of yl is read by no one: its readers have passed this barrier's last turn
#pragma unroll
            for (int i = 0; i < SC; ++i) {
                if (i % a.ntiles != w.nt || t + i >= w.end || !w.in) continue;
                float o = skip * value<BF16>(xr[i]);
                for (int k = 0; k < a.ntiles; ++k) o += yl[par][k][i][w.lane];
                if constexpr (HASZ) {
                    const float z = value<BF16>(zr[i]);
                    o *= z * sigmoid(z);
                }
                put<BF16>(const_cast<char*>(row<BF16>(a.y, (w.b * a.T + t + i) * a.D)), w.c, o);
            }
            par ^= 1;
        }
    }
    if constexpr (EMIT) {
        if (w.nt == 0 && w.in)
            for (int64_t t = w.end > w.t0 ? w.end : w.t0; t < w.t1; ++t)
                put<BF16>(const_cast<char*>(row<BF16>(a.y, (w.b * a.T + t) * a.D)), w.c, 0.f);
        if (a.S && w.seg == a.nseg - 1) store_dn(a, w, a.S + w.b * per, h);
    } else {
        store_tile(a.ends + (w.seg * waves + wave) * 1024, w.lane, h);
        if (w.nt == 0) a.steps[(w.seg * a.tiles + w.tile) * 64 + w.lane] = steps;
    }
}

template <bool BF16, bool HASZ, bool EMIT>
void sel_go(const SelArgs& a, int nseg, hipStream_t st) {
    const dim3 grid((unsigned)a.tiles, (unsigned)nseg);
    if (a.ntiles > 1) hipLaunchKernelGGL((sel_kernel<BF16, HASZ, true, EMIT>), grid, dim3(64 * a.ntiles), 0, st, a);
    else hipLaunchKernelGGL((sel_kernel<BF16, HASZ, false, EMIT>), grid, dim3(64), 0, st, a);
}

// Segments: enough wavefronts for the SIMDs, of at least 64 tokens
void sel_split(int64_t B, int64_t T, int G, int D, int N, int64_t* L, int* nseg) {
    const int64_t waves = sel_tiles(B, G, D) * sel_ntiles(N), want = (4096 + waves - 1) / waves;
    int64_t len = (T + want - 1) / want;
    if (len < 64) len = 64;
    if (len > T) len = T > 0 ? T : 1;
    len = (len + SC - 1) / SC * SC;
    *L = len;
    *nseg = T > len ? (int)((T + len - 1) / len) : 1;
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
        a.bf16 ? sel_go<true, false, false>(a, a.nseg - 1, st) : sel_go<false, false, false>(a, a.nseg - 1, st);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        SelCarryArgs c{};
        c.ends = a.ends; c.steps = a.steps; c.A = a.A; c.from = a.S0;
        c.tiles = a.tiles; c.nseg = a.nseg; c.ntiles = a.ntiles; c.ctiles = a.ctiles; c.G = a.G; c.D = a.D; c.N = a.N;
        if ((e = sel_carry(c, c, 1, st)) != hipSuccess) return e;
    }
    if (a.z) a.bf16 ? sel_go<true, true, true>(a, a.nseg, st) : sel_go<false, true, true>(a, a.nseg, st);
    else a.bf16 ? sel_go<true, false, true>(a, a.nseg, st) : sel_go<false, false, true>(a, a.nseg, st);
    return hipGetLastError();
}

}  // namespace sdm
