// selective_bwd.hip -- the gradients of the selective state-space scan (selective.hip) on gfx950. With
// gy_t = dy_t silu(z_t), u_t = delta_t x_t, a_t = exp(delta_t A) and g_t = C_t gy_t + a_{t+1} g_{t+1} (behind the
// last token dL/dh):
//   dC_t = sum_d gy_t h_t             dB_t = sum_d u_t g_t
//   dx_t = D gy_t + delta_t sum_n g_t B_t
//   ddelta_t = sum_n A g_t a_t h_{t-1} + x_t sum_n g_t B_t,   ddt_t = ddelta_t sigmoid(dt_t + bias)
//   dz_t = dy_t (C_t h_t + D x_t) silu'(z_t)
//   dA = sum_t delta_t g_t a_t h_{t-1},   dD = sum_t gy_t x_t,   dbias = sum_t ddt_t,   dS0 = a_1 g_1
//
// Nothing is kept from the forward call. A first pass over the segments forms the states again, from zeros,
// leaves one every 8 tokens (with the sum of steps since the segment's start, by whose decay the segment's
// own starting state is added), and sums what a segment passes to the one before it. Carries run through the
// segments both ways. The last pass walks the chunks backwards, half a chunk (4 tokens) at a time: it forms
// the 4 states again, keeping each token's decay in registers and its decayed state in LDS, and then walks them back.
// Sums over channels leave a row a tile, added by a last pass.
//
// Bound by vector instructions (335 a token and tile in the last pass, 123 in the first; issued in 84 and 80% of the cycles,
// at 2 and 4 wavefronts a SIMD): 4 x 4096 x 2048 with 16 states in bf16, first pass 163 to 174 us, carries 15, last pass 403 to 431,
// sums 28 (610 a call), for 92 us of HBM at a copy's rate. (A state every 4 tokens instead would spare forming 4 states of 8 twice, a tenth
// of the last pass, but the first one has no room for 268 MB more: it moves 606 MB as it is.)
#include <cmath>
#include <type_traits>

#include "selective.h"

namespace sdm {
namespace {

constexpr int HC = SC / 2;

template <bool BF16, bool HASZ>
__global__ __launch_bounds__(256, 4) void sel_ends_kernel(SelBwdArgs a) {
    __shared__ float4 fan[4][HC][16];  // half a chunk's steps: a lane's 4 channels side by side
    const SelAt w = sel_at<BF16>(a);
    const f32x16 a2 = load_dn(a, w, a.A, 1.44269504f);
    const int64_t wave = w.tile * a.ntiles + w.nt, waves = a.tiles * a.ntiles;
    float4(*dl)[16] = fan[w.nt];
    const char* px = row<BF16>(a.x, w.b * a.x_b);
    const char* pd = row<BF16>(a.dt, w.b * a.dt_b);
    const char* pz = HASZ ? row<BF16>(a.z, w.b * a.z_b) : nullptr;
    const char* py = row<BF16>(a.dy, w.b * a.dy_b);
    const char* pB = row<BF16>(a.Bm, w.b * a.B_b + w.g * a.B_g);
    const char* pC = row<BF16>(a.Cm, w.b * a.C_b + w.g * a.C_g);
    const float bias = a.bias ? a.bias[w.c] : 0.f;
    const uint8_t* start = a.start ? a.start + w.b * a.T : nullptr;
    f32x16 h = zeros16(), g = zeros16(), p;
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = 1.f;
    float steps = 0.f;
    bool cut = false;  // a sequence began in the segment: nothing crosses it
    int64_t half = w.seg * (a.L / HC);
    for (int64_t t = w.t0; t < w.end; t += HC, ++half) {
        const int64_t left = w.end - t;
        if (half % 2 == 0) {
            store_tile(a.marks + (half / 2 * waves + wave) * 1024, w.lane, h);
            if (w.nt == 0) a.msteps[(half / 2 * a.tiles + w.tile) * 64 + w.lane] = cut ? GONE : steps;
        }
        const Rows<BF16> X(px, a.x_t, t), T(pd, a.dt_t, t), Z(pz, HASZ ? a.z_t : 0, HASZ ? t : 0), Y(py, a.dy_t, t);
        const Rows<BF16> B(pB, a.B_t, t), C(pC, a.C_t, t);
        uint32_t xr[HC], dr[HC], zr[HC], yr[HC];
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            xr[i] = X.get(w.vo, upto(i, left));
            dr[i] = T.get(w.vo, upto(i, left));
            yr[i] = Y.get(w.vo, upto(i, left));
            if constexpr (HASZ) zr[i] = Z.get(w.vo, upto(i, left));
        }
        const uint32_t st = starts(start, t, w.end, w.lane);
        float bq[4], cq[4];
        spread(load_bc(B, w, 0, left, a.N), bq);
        spread(load_bc(C, w, 0, left, a.N), cq);
        float u[HC], gy[HC];
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            const bool on = w.in && i < left;  // (a lane without a channel adds nothing: its states go into the sums below times 0)
            float delta = step_of(value<BF16>(dr[i]) + bias, a.softplus);
            u[i] = on ? delta * value<BF16>(xr[i]) : 0.f;
            delta = i < left ? delta : 0.f;
            steps += delta;
            gy[i] = value<BF16>(yr[i]);
            if constexpr (HASZ) {
                const float z = value<BF16>(zr[i]);
                gy[i] *= z * sigmoid(z);
            }
            cut |= (st >> i & 1u) != 0;
            gy[i] = on && !cut ? gy[i] : 0.f;
            cq[i] = cut ? 0.f : cq[i];
            reinterpret_cast<float*>(dl[i])[4 * w.j + w.q] = st >> i & 1u ? 0.f : delta;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            const f32x16 d = decays(dl[i][w.j], a2, st >> i & 1u ? GONE : 0.f), cg = outer_add(cq[i], gy[i], zeros16());
            decay(h, d);
            h = outer_add(bq[i], u[i], h);
            decay(p, d);
#pragma unroll
            for (int k = 0; k < 16; ++k) g[k] = fmaf(p[k], cg[k], g[k]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const int64_t at = (w.seg * waves + wave) * 1024;
    store_tile(a.ends + at, w.lane, h);
    store_tile(a.gends + at, w.lane, g);
    if (w.nt == 0) a.steps[(w.seg * a.tiles + w.tile) * 64 + w.lane] = cut ? GONE : steps;
}

// Lane j of a row of 16 lanes gets the row's sum of v[j / 4]
__device__ __forceinline__ float row_sums(const float (&v)[4], int j) {
    const bool hi = j & 8, odd = j & 4;
    float s0 = (hi ? v[2] : v[0]) + dpp<0x128>(hi ? v[0] : v[2]);  // row_ror:8
    float s1 = (hi ? v[3] : v[1]) + dpp<0x128>(hi ? v[1] : v[3]);
    float s = (odd ? s1 : s0) + dpp<0x141>(odd ? s0 : s1);         // row_half_mirror: lane 7 - j of the half row
    s += dpp<0x4E>(s);                                             // quad_perm 2,3,0,1
    return s + dpp<0xB1>(s);                                       // quad_perm 1,0,3,2
}

// LDS of a wavefront, in floats: half a chunk's decayed states a_t h_{t-1}, its B and C, and its steps, inputs and
// gradients (with several tiles of states, in their place, the sums over states that the wavefronts exchange)
constexpr int KEPT = HC * 1024, FAN = KEPT + 2 * HC * 16, SHARE = FAN + 3 * HC * 64;
static_assert(8 * SHARE * 4 <= 160 * 1024, "8 wavefronts a CU");

template <bool BF16, bool HASZ, bool MULTI>
__global__ __launch_bounds__(MULTI ? 256 : 64, 2) void sel_grads_kernel(SelBwdArgs a) {
    extern __shared__ float4 lds4[];
    const SelAt w = sel_at<BF16>(a);
    const int NT = MULTI ? a.ntiles : 1;
    float* mine = reinterpret_cast<float*>(lds4) + w.nt * SHARE;
    float4* kept = reinterpret_cast<float4*>(mine);
    float(*bl)[16] = reinterpret_cast<float(*)[16]>(mine + KEPT);
    float(*cl)[16] = bl + HC;
    float* fan = mine + FAN;  // [HC][3][64]: a channel's values at 4 j + blk, so that a lane reads its 4 channels' at once
    const f32x16 a2 = load_dn(a, w, a.A, 1.44269504f);
    const int64_t wave = w.tile * a.ntiles + w.nt, waves = a.tiles * a.ntiles, per = (int64_t)a.D * a.N;
    const char* px = row<BF16>(a.x, w.b * a.x_b);
    const char* pd = row<BF16>(a.dt, w.b * a.dt_b);
    const char* pz = HASZ ? row<BF16>(a.z, w.b * a.z_b) : nullptr;
    const char* py = row<BF16>(a.dy, w.b * a.dy_b);
    const char* pB = row<BF16>(a.Bm, w.b * a.B_b + w.g * a.B_g);
    const char* pC = row<BF16>(a.Cm, w.b * a.C_b + w.g * a.C_g);
    const char* pdx = row<BF16>(a.dx, w.b * a.T * a.D);
    const char* pdd = row<BF16>(a.ddt, w.b * a.T * a.D);
    const char* pdz = HASZ ? row<BF16>(a.dz, w.b * a.T * a.D) : nullptr;
    const char* pbc = row<false>(a.part_bc, (((w.c0 / 64) * a.B + w.b) * a.G + w.g) * a.T * NT * 32 + w.nt * 32);
    // the lane's element of a token's 16 sums for dB and 16 for dC
    const uint32_t vbc = (w.j & 3) < 2 ? 4u * ((w.j & 1) * 16 + 4 * w.q + (w.j >> 2)) : OOB;
    const float bias = a.bias ? a.bias[w.c] : 0.f, skip = a.Dskip ? a.Dskip[w.c] : 0.f;
    const uint8_t* start = a.start ? a.start + w.b * a.T : nullptr;
    const int64_t at = (w.seg * waves + wave) * 1024;
    f32x16 g = load_tile(a.gends + at, w.lane), dA = zeros16();
    float dD = 0.f, dbias = 0.f;
    // behind the last token: gradients of 0
    if (w.nt == 0)
        for (int64_t t = w.end > w.t0 ? w.end : w.t0; t < w.t1; ++t) {
            Rows<BF16>(pdx, a.D, t).put(w.vput, 0, 0.f);
            Rows<BF16>(pdd, a.D, t).put(w.vput, 0, 0.f);
            if constexpr (HASZ) Rows<BF16>(pdz, a.D, t).put(w.vput, 0, 0.f);
        }
    const int64_t chunks = w.end > w.t0 ? (w.end - w.t0 + SC - 1) / SC : 0, first = w.seg * (a.L / SC);
    // A chunk's 8 tokens, or the first `left` of them
    auto chunk = [&](auto whole, int64_t ch, int64_t left) {
        constexpr bool ALL = decltype(whole)::value;
        const int64_t t = w.t0 + ch * SC;
        const Rows<BF16> X(px, a.x_t, t), T(pd, a.dt_t, t), Z(pz, HASZ ? a.z_t : 0, HASZ ? t : 0), Y(py, a.dy_t, t);
        const Rows<BF16> B(pB, a.B_t, t), C(pC, a.C_t, t);
        uint32_t xr[SC], dr[SC], zr[SC], yr[SC];
        float bv[2], cv[2];
#pragma unroll
        for (int i = 0; i < SC; ++i) {
            const uint32_t m = ALL ? i : upto(i, left);
            xr[i] = X.get(w.vo, m);
            dr[i] = T.get(w.vo, m);
            yr[i] = Y.get(w.vo, m);
            if constexpr (HASZ) zr[i] = Z.get(w.vo, m);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            bv[k] = load_bc(B, w, k, left, a.N);
            cv[k] = load_bc(C, w, k, left, a.N);
        }
        const uint32_t st = starts(start, t, w.end, w.lane);
        // the state in front of the chunk
        f32x16 h0 = load_tile(a.marks + ((first + ch) * waves + wave) * 1024, w.lane);
        {
            const float* ms = a.msteps + ((first + ch) * a.tiles + w.tile) * 64 + w.j;
            const f32x16 hs = load_tile(a.ends + at, w.lane);
            const float s4[4] = {ms[0], ms[16], ms[32], ms[48]};
            __builtin_amdgcn_sched_barrier(0);  // all of the chunk's loads in flight before the first one is waited for
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float s = s4[k];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = fmaf(__builtin_amdgcn_exp2f(a2[4 * k + r] * s), hs[4 * k + r], h0[4 * k + r]);
                    h0[4 * k + r] = s == GONE ? h0[4 * k + r] : e;
                }
            }
        }
        f32x16 h = h0;
        if (ALL || left > HC) {  // and in front of its second half
            float bq[4];
            spread(bv[0], bq);
#pragma unroll
            for (int i = 0; i < HC; ++i) {
                const float delta = step_of(value<BF16>(dr[i]) + bias, a.softplus);
                const bool begins = st >> i & 1u;
                float d4[4];
                spread(begins ? 0.f : delta, d4);
                decay(h, decays(make_float4(d4[0], d4[1], d4[2], d4[3]), a2, begins ? GONE : 0.f));
                h = outer_add(bq[i], w.in ? delta * value<BF16>(xr[i]) : 0.f, h);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int half = 1; half >= 0; --half) {
            if (!ALL && half * HC >= left) continue;
            if (half == 0) h = h0;
            bl[w.q][w.j] = bv[half];
            cl[w.q][w.j] = cv[half];
            float bq[4], cq[4], delta[HC], gy[HC], u[HC];
            spread(bv[half], bq);
            spread(cv[half], cq);
            // a token's step and output gradient (0 where it is not there; no gradient of a channel that is not there)
            auto token = [&](int i) {
                const int m = half * HC + i;
                const bool there = ALL || m < left;
                const float de = step_of(value<BF16>(dr[m]) + bias, a.softplus);
                delta[i] = there ? de : 0.f;
                float y = value<BF16>(yr[m]);
                if constexpr (HASZ) {
                    const float z = value<BF16>(zr[m]);
                    y *= z * sigmoid(z);
                }
                gy[i] = w.in && there ? y : 0.f;
            };
#pragma unroll
            for (int i = 0; i < HC; ++i) {
                token(i);
                u[i] = w.in && (ALL || half * HC + i < left) ? delta[i] * value<BF16>(xr[half * HC + i]) : 0.f;
                float* f = fan + i * 192 + 4 * w.j + w.q;
                f[0] = st >> (half * HC + i) & 1u ? 0.f : delta[i];  // (behind a begin there is no state for dA either)
                f[64] = u[i];
                f[128] = gy[i];
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            auto fanned = [&](int i, int what, float (&o)[4]) {
                const float4 v = *reinterpret_cast<const float4*>(fan + i * 192 + what * 64 + 4 * w.j);
                o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
            };
            f32x16 dec[HC];  // a_t
#pragma unroll
            for (int i = 0; i < HC; ++i) {
                dec[i] = decays(*reinterpret_cast<const float4*>(fan + i * 192 + 4 * w.j), a2, st >> (half * HC + i) & 1u ? GONE : 0.f);
                decay(h, dec[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    kept[(i * 4 + k) * 64 + w.lane] = make_float4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
                if (i < HC - 1) h = outer_add(bq[i], u[i], h);
                __builtin_amdgcn_sched_barrier(0);
            }
            // a token's own gradients, from the sums over its states
            auto finish = [&](int i, float sa, float sb, float sc) {
                const int m = half * HC + i;
                const float x = value<BF16>(xr[m]);
                float dd = fmaf(x, sb, 0.69314718f * sa);
                const float sg = sigmoid(value<BF16>(dr[m]) + bias);
                dd *= a.softplus ? sg : 1.f;
                if (!ALL) dd = m < left ? dd : 0.f;
                dbias += dd;
                dD = fmaf(gy[i], x, dD);
                const uint32_t vo = ALL || m < left ? w.vput : OOB;
                Rows<BF16>(pdx, a.D, t).put(vo, m, fmaf(delta[i], sb, skip * gy[i]));
                Rows<BF16>(pdd, a.D, t).put(vo, m, dd);
                if constexpr (HASZ) {
                    const float z = value<BF16>(zr[m]), s = sigmoid(z);
                    Rows<BF16>(pdz, a.D, t).put(vo, m, value<BF16>(yr[m]) * fmaf(skip, x, sc) * s * fmaf(z, 1.f - s, 1.f));
                }
            };
#pragma unroll
            for (int i = HC - 1; i >= 0; --i) {
                const int m = half * HC + i;
                g = outer_add(cq[i], gy[i], g);
                const float4 bn = *reinterpret_cast<const float4*>(&bl[i][4 * w.q]);
                const float4 cn = *reinterpret_cast<const float4*>(&cl[i][4 * w.q]);
                const float b4[4] = {bn.x, bn.y, bn.z, bn.w}, c4[4] = {cn.x, cn.y, cn.z, cn.w};
                float ds[4], us[4], gs[4], sb[4] = {}, sc[4] = {}, pb[4], pa[4], pc[4];
                fanned(i, 0, ds);
                fanned(i, 1, us);
                fanned(i, 2, gs);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 kp = kept[(i * 4 + k) * 64 + w.lane];
                    const float k4[4] = {kp.x, kp.y, kp.z, kp.w};
                    pa[k] = pb[k] = pc[k] = 0.f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int e = 4 * k + r;
                        const float hv = fmaf(us[k], b4[r], k4[r]), gk = g[e] * k4[r];
                        sb[r] = fmaf(us[k], g[e], sb[r]);
                        sc[r] = fmaf(gs[k], hv, sc[r]);
                        pa[k] = fmaf(a2[e], gk, pa[k]);
                        pb[k] = fmaf(b4[r], g[e], pb[k]);
                        if constexpr (HASZ) pc[k] = fmaf(c4[r], hv, pc[k]);
                        dA[e] = fmaf(ds[k], gk, dA[e]);
                        g[e] = sdm_mul_zero(dec[i][e], g[e]);
                    }
                }
                const float qa = gather_sum(pa), qb = gather_sum(pb), qc = HASZ ? gather_sum(pc) : 0.f;
                const float rb = row_sums(sb, w.j), rc = row_sums(sc, w.j);
                Rows<false>(pbc, NT * 32, t).put(ALL || m < left ? vbc : OOB, m, w.j & 1 ? rc : rb);
                if constexpr (MULTI) {
                    float* s = fan + i * 192 + w.lane;  // token i's values there have been read
                    s[0] = qa;
                    s[64] = qb;
                    s[128] = qc;
                } else {
                    finish(i, qa, qb, qc);
                }
                __builtin_amdgcn_sched_barrier(0x100);
            }
            if constexpr (MULTI) {
                const float* all = reinterpret_cast<const float*>(lds4);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < HC; ++i) {
                    if (i % a.ntiles != w.nt) continue;
                    float s[3] = {};
                    const int at8 = half * HC + i;
                    const uint32_t m8 = ALL ? at8 : upto(at8, left);  // (again, out of the cache: kept, they would not fit the registers)
                    xr[at8] = X.get(w.vo, m8);
                    dr[at8] = T.get(w.vo, m8);
                    yr[at8] = Y.get(w.vo, m8);
                    if constexpr (HASZ) zr[at8] = Z.get(w.vo, m8);
                    for (int k = 0; k < a.ntiles; ++k)
#pragma unroll
                        for (int m = 0; m < 3; ++m) s[m] += all[k * SHARE + FAN + i * 192 + m * 64 + w.lane];
                    token(i);
                    finish(i, s[0], s[1], s[2]);
                }
                __syncthreads();  // before the next sums
            }
        }
    };
    int64_t ch = chunks - 1;
    if (ch >= 0 && w.end - w.t0 < chunks * SC) {
        chunk(std::false_type{}, ch, w.end - w.t0 - ch * SC);
        --ch;
    }
    for (; ch >= 0; --ch) chunk(std::true_type{}, ch, SC);
    store_tile(a.part_A + at, w.lane, dA);
    if (a.dS0 && w.seg == 0) store_dn(a, w, a.dS0 + w.b * per, g);
    float* pd2 = a.part_D + ((w.seg * a.ntiles + w.nt) * a.tiles + w.tile) * 128 + w.lane;
    pd2[0] = dD;
    pd2[64] = dbias;
}

// dB and dC [B,T,G,N]: the sums of the channel tiles' rows, in 64 bits and in their order; 0 behind the last token
__global__ __launch_bounds__(256) void sel_bc_kernel(SelBwdArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, cols = a.B * a.G * a.T * a.ntiles * 32;  // [b][g][t][nt][2][16]
    if (i >= cols) return;
    const int64_t u = i / (a.ntiles * 32);
    const int m = (int)(i % (a.ntiles * 32)), n = m / 32 * 16 + (m & 15);
    const int64_t t = u % a.T, bg = u / a.T, b = bg / a.G, g = bg % a.G;
    if (n >= a.N) return;
    double s = 0.0;
    if (!a.lengths || t < a.lengths[b])
#pragma unroll 8
        for (int k = 0; k < a.ctiles; ++k) s += a.part_bc[k * cols + i];
    (m & 16 ? a.dC : a.dB)[((b * a.T + t) * a.G + g) * a.N + n] = (float)s;
}

// dA [D][N] of the columns [g][ct][nt][blk][lane][r]
struct SelSumA {
    float* dA;
    int G, D, N, ctiles, ntiles;
    __device__ void operator()(int64_t i, float v) const {
        const int r = (int)(i & 3), lane = (int)(i >> 2 & 63), blk = (int)(i >> 8 & 3);
        int64_t w = i >> 10;
        const int n = (int)(w % ntiles) * 16 + 4 * (lane >> 4) + r;
        w /= ntiles;
        const int c = (int)(w % ctiles) * 64 + 16 * blk + (lane & 15), g = (int)(w / ctiles);
        if (c < D / G && n < N) dA[(int64_t)(g * (D / G) + c) * N + n] = v;
    }
};
// dD and dbias [D] of the columns [g][ct][2][64]
struct SelSumD {
    float* dD; float* dbias;
    int G, D, ctiles;
    __device__ void operator()(int64_t i, float v) const {
        const int c = (int)((i >> 7) % ctiles) * 64 + (int)(i & 63), g = (int)((i >> 7) / ctiles);
        float* o = i & 64 ? dbias : dD;
        if (o && c < D / G) o[g * (D / G) + c] = v;
    }
};

// The launches are the same for one segment: any is cut (64 tokens of one sequence: 107 -> 45 us), into twice what fits.
// A segment's sums for dA, dD and dt_bias are one chain of fp32 additions, up to n / 2 half steps off in n like terms, so
// it has 1024 tokens at most, or the root of T / 10 (more in 10^7 tokens and up, and fewer than 2^16 segments of 2^27).
// 64 x 4096 x 2048 with 16 states, bf16: 9.5 ms by one segment of 2048 tokens a wavefront, 9.3 so.
void sel_bwd_split(int64_t B, int64_t T, int G, int D, int N, int64_t* L, int* nseg) {
    sel_segments(B, T, G, D, N, 4096, L, nseg);
    int64_t most = ((int64_t)sqrt(0.1 * (double)T) + SC - 1) / SC * SC;
    if (most < 1024) most = 1024;
    if (*L > most) {
        *L = most;
        *nseg = (int)((T + most - 1) / most);
    }
}

// The workspace's parts, in floats
struct SelBwdParts {
    int64_t ends, gends, steps, marks, msteps, part_bc, part_A, part_D, end;
};
SelBwdParts sel_bwd_parts(int64_t B, int64_t T, int G, int D, int N, int64_t L, int nseg) {
    const int64_t tiles = sel_tiles(B, G, D), nt = sel_ntiles(N), tile = tiles * nt * 1024, chunks = nseg * (L / SC);
    SelBwdParts p;
    p.ends = 0;
    p.gends = p.ends + nseg * tile;
    p.steps = p.gends + nseg * tile;
    p.marks = p.steps + nseg * tiles * 64;
    p.msteps = p.marks + chunks * tile;
    p.part_bc = p.msteps + chunks * tiles * 64;
    p.part_A = p.part_bc + tiles * T * nt * 32;
    p.part_D = p.part_A + nseg * tile;
    p.end = p.part_D + nseg * nt * tiles * 128;
    return p;
}

template <bool BF16, bool HASZ>
hipError_t sel_bwd_grads(const SelBwdArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)a.tiles, (unsigned)a.nseg);
    if (a.ntiles == 1) {
        hipLaunchKernelGGL((sel_grads_kernel<BF16, HASZ, false>), grid, dim3(64), SHARE * 4, st, a);
    } else {
        const int bytes = a.ntiles * SHARE * 4;  // up to 80 KB
        hipLaunchKernelGGL((sel_grads_kernel<BF16, HASZ, true>), grid, dim3(64 * a.ntiles), bytes, st, a);
    }
    return hipGetLastError();
}
template <bool BF16, bool HASZ>
void sel_bwd_ends(const SelBwdArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((sel_ends_kernel<BF16, HASZ>), dim3((unsigned)a.tiles, (unsigned)a.nseg), dim3(64 * a.ntiles), 0, st, a);
}

}  // namespace

int64_t selective_backward_workspace_bytes(int64_t B, int64_t T, int G, int D, int N) {
    int64_t L;
    int nseg;
    sel_bwd_split(B, T, G, D, N, &L, &nseg);
    return sel_bwd_parts(B, T, G, D, N, L, nseg).end * 4;
}

hipError_t launch_selective_backward(SelBwdArgs a, hipStream_t st) {
    a.ctiles = sel_ctiles(a.G, a.D);
    a.ntiles = sel_ntiles(a.N);
    a.tiles = sel_tiles(a.B, a.G, a.D);
    sel_bwd_split(a.B, a.T, a.G, a.D, a.N, &a.L, &a.nseg);
    const SelBwdParts p = sel_bwd_parts(a.B, a.T, a.G, a.D, a.N, a.L, a.nseg);
    float* ws = static_cast<float*>(a.workspace);
    a.ends = ws + p.ends; a.gends = ws + p.gends; a.steps = ws + p.steps; a.marks = ws + p.marks; a.msteps = ws + p.msteps;
    a.part_bc = ws + p.part_bc; a.part_A = ws + p.part_A; a.part_D = ws + p.part_D;
    if (a.z) a.bf16 ? sel_bwd_ends<true, true>(a, st) : sel_bwd_ends<false, true>(a, st);
    else a.bf16 ? sel_bwd_ends<true, false>(a, st) : sel_bwd_ends<false, false>(a, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    SelCarryArgs c{};
    c.ends = a.ends; c.steps = a.steps; c.A = a.A; c.from = a.S0;
    c.tiles = a.tiles; c.nseg = a.nseg; c.ntiles = a.ntiles; c.ctiles = a.ctiles; c.G = a.G; c.D = a.D; c.N = a.N;
    SelCarryArgs r = c;
    r.ends = a.gends; r.from = a.dS; r.rev = true;
    if ((e = sel_carry(c, r, 2, st)) != hipSuccess) return e;
    if (a.z) e = a.bf16 ? sel_bwd_grads<true, true>(a, st) : sel_bwd_grads<false, true>(a, st);
    else e = a.bf16 ? sel_bwd_grads<true, false>(a, st) : sel_bwd_grads<false, false>(a, st);
    if (e != hipSuccess) return e;
    const int64_t cols = a.B * a.G * a.T * a.ntiles * 32, bg = (int64_t)a.G * a.ctiles;
    if (cols > 0) {
        hipLaunchKernelGGL(sel_bc_kernel, dim3((unsigned)((cols + 255) / 256)), dim3(256), 0, st, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    e = sum_columns(a.part_A, a.nseg * a.B, bg * a.ntiles * 1024, SelSumA{a.dA, a.G, a.D, a.N, a.ctiles, a.ntiles}, st);
    if (e != hipSuccess) return e;
    return sum_columns(a.part_D, a.nseg * a.ntiles * a.B, bg * 128, SelSumD{a.dD, a.dbias, a.G, a.D, a.ctiles}, st);
}

}  // namespace sdm
