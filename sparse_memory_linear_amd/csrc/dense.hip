// dense.hip -- the dense gated recurrence on gfx950: a d_k x d_v state per head
// in which every token decays all rows and adds one outer product,
//   S_t = alpha_t S_{t-1} + beta_t k_t (x) v_t,     y_t = q_t S_t,
// and its gradients. The sparse scan's dense counterpart: same gates, v and y.
//
// One recurrence serves the forward and every gradient. With rows xi, kap (DK
// wide) and omg (DV wide), processed forwards or backwards in t,
//   X_u = a_u X_{u-1} + b_u kap_u (x) omg_u,    out_u = o_u xi_u X_u:
//   y   forwards:  kap = k,  omg = v,  xi = q,  X = S,   a_u = alpha_t, b = beta
//   dq  forwards:  kap = v,  omg = k,  xi = dy, X = S^T, a_u = alpha_t, b = beta
//   dk  backwards: kap = dy, omg = q,  xi = v,  X = G^T, a_u = alpha_{t+1}, o = beta
//   dv  backwards: kap = q,  omg = dy, xi = k,  X = G,   a_u = alpha_{t+1}, o = beta
// with G_t = alpha_{t+1} G_{t+1} + q_t (x) dy_t (the state's gradient; past the
// end it is dL/dS_T, undecayed). d/dbeta_t = k_t . (dk_t / beta_t), and
// E_t = dL/d ln alpha_t = <G_t, alpha_t S_{t-1}> follows from
//   E_t = E_{t+1} + q_t . dq_t - k_t . dk_t,
// started at each segment's end from <alpha_{t+1} G_{t+1}, S_t> there, so that
// no sum runs over more than one segment.
//
// Chunks: a workgroup carries a slab of X in registers over a segment's tokens,
// C at a time. Within a chunk, with D_ts = a_{s+1} .. a_t,
//   out = o (pre X_start + (tril(xi kap^T) . D . b) omg),  pre_t = a_c0 .. a_t
//   X_end = total X_start + sum_s kap_s (x) (D_end,s b_s omg_s).
// The decays are products of the gates, never quotients or differences of
// logarithms: a gate of 0 gives exact zeros and no 0/0. A 16 x 16 block of D on
// the diagonal is kept whole; off it, D_ts is the product from t's block start,
// the whole blocks between, and to s's block end.
//
// Segments: with few streams the tokens are split into segments; a pass leaves
// each segment's own sum, a second adds them up over the segments (giving each
// one's starting state), and the last computes the outputs.
#include "sdm_buffer.h"
#include "sdm_internal.h"

namespace sdm {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;

constexpr int DENSE_SLAB = 64;  // columns of X per workgroup: 16 per wavefront

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// 8 consecutive elements (index e, a multiple of 8) as fp32
__device__ __forceinline__ void load8(const void* p, bool bf16, int64_t e, float (&v)[8]) {
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e);
        v[0] = bf_lo(u.x); v[1] = bf_hi(u.x); v[2] = bf_lo(u.y); v[3] = bf_hi(u.y);
        v[4] = bf_lo(u.z); v[5] = bf_hi(u.z); v[6] = bf_lo(u.w); v[7] = bf_hi(u.w);
    } else {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
        const float4 x = f[0], y = f[1];
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    }
}

__device__ __forceinline__ float load1(const void* p, bool bf16, int64_t e) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[e] << 16) : static_cast<const float*>(p)[e];
}

// The chunk's decays, by one wavefront: lane l < C holds its step's gate.
template <int C>
struct Decay {
    float diag[C / 16][16][16];  // D_ts within a block of 16 (0 above the diagonal)
    float pre[C];                // gates from the block's start through t
    float suf[C];                // gates after s through the block's end
    float tot[C / 16];           // a block's gates
    float gate[C];
    float in[C];                 // b_s
    __device__ __forceinline__ float before(int t) const {  // from the chunk's start through t
        float p = pre[t];
        for (int b = 0; b < t >> 4; ++b) p *= tot[b];
        return p;
    }
    __device__ __forceinline__ float after(int s) const {   // after s through the chunk's end
        float p = suf[s];
        for (int b = (s >> 4) + 1; b < C / 16; ++b) p *= tot[b];
        return p;
    }
    __device__ __forceinline__ float total() const {
        float p = tot[0];
        for (int b = 1; b < C / 16; ++b) p *= tot[b];
        return p;
    }
};

// DKT: 16-row tiles of X (DK padded with zeros); C: tokens per chunk.
// OUT false: only the state at the segment's end (starting from zero).
template <int DKT, int C, bool OUT>
__global__ __launch_bounds__(256) void dense_kernel(DenseArgs a) {
    constexpr int DKP = DKT * 16, SV = DENSE_SLAB, NT = C / 16;
    constexpr int LK = DKP + 4, LV = SV + 4, LP = C + 4;
    extern __shared__ float lds[];
    float* Ka = lds;                         // [C][LK]
    float* Om = Ka + C * LK;                 // [C][LV]
    float* Xi = Om + C * LV;                 // [C][LK] (OUT)
    float* P = Xi + (OUT ? C * LK : 0);      // [C][LP] (OUT)
    __shared__ Decay<C> dc;
    __shared__ float dots[4][C];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m16 = lane & 15, g4 = lane >> 4;
    const int64_t u = blockIdx.x;
    const int slab = (int)(u % a.nslab), seg = (int)(u / a.nslab % a.nseg);
    const int64_t s = u / a.nslab / a.nseg;  // stream
    const int64_t lo = (int64_t)seg * a.L, hi = lo + a.L < a.T ? lo + a.L : a.T;
    const int c0 = slab * SV, col = c0 + w * 16 + m16;
    const bool col_ok = col < a.DV;
    const int64_t row0 = s * a.T;
    const int64_t st0 = (seg * a.NS + s) * (int64_t)a.DK * a.DV;

    f32x4_t X[DKT];
#pragma unroll
    for (int k = 0; k < DKT; ++k) {
        X[k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (OUT && a.X0) {
            const int64_t base = a.X0_seg ? st0 : s * (int64_t)a.DK * a.DV;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = k * 16 + 4 * g4 + i;
                if (r < a.DK && col_ok) X[k][i] = a.X0[base + r * (int64_t)a.x_row + col * (int64_t)a.x_col];
            }
        }
    }
    float segdec = 1.f;
    for (int64_t c = lo; c < hi; c += C) {  // step numbers; token of step c + j below
        const int n = (int)(hi - c < C ? hi - c : C);
        auto token = [&](int j) { return a.rev ? lo + hi - 1 - (c + j) : c + j; };
        __syncthreads();
        if (w == 0) {
            if (lane < C) {
                float g = 1.f, b = 0.f;
                if (lane < n) {
                    const int64_t t = token(lane);
                    if (!a.rev) g = a.a[row0 + t];
                    else if (t + 1 < a.T) g = a.a[row0 + t + 1];
                    b = a.b ? a.b[row0 + t] : 1.f;
                }
                dc.gate[lane] = g;
                dc.in[lane] = b;
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (lane < C) {
                const int blk = lane >> 4, j = lane & 15;
                float p = 1.f;
                for (int t = 0; t < 16; ++t) {
                    if (t > j) p *= dc.gate[blk * 16 + t];
                    dc.diag[blk][t][j] = t < j ? 0.f : p;
                }
                dc.suf[lane] = p;
                float f = 1.f;
                for (int t = 0; t <= j; ++t) f *= dc.gate[blk * 16 + t];
                dc.pre[lane] = f;
                if (j == 15) dc.tot[blk] = f;
            }
        }
        for (int e = tid; e < C * (DKP / 8); e += 256) {
            const int j = e / (DKP / 8), q = e % (DKP / 8) * 8;
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, k[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (j < n && q < a.DK) {
                const int64_t at = (row0 + token(j)) * a.DK + q;
                load8(a.kap, a.kap_bf16, at, k);
                if (OUT) load8(a.xi, a.xi_bf16, at, x);
            }
            *reinterpret_cast<float4*>(&Ka[j * LK + q]) = make_float4(k[0], k[1], k[2], k[3]);
            *reinterpret_cast<float4*>(&Ka[j * LK + q + 4]) = make_float4(k[4], k[5], k[6], k[7]);
            if (OUT) {
                *reinterpret_cast<float4*>(&Xi[j * LK + q]) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(&Xi[j * LK + q + 4]) = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
        for (int e = tid; e < C * (SV / 8); e += 256) {
            const int j = e / (SV / 8), q = e % (SV / 8) * 8;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (j < n && c0 + q < a.DV) load8(a.omg, a.omg_bf16, (row0 + token(j)) * a.DV + c0 + q, v);
            *reinterpret_cast<float4*>(&Om[j * LV + q]) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(&Om[j * LV + q + 4]) = make_float4(v[4], v[5], v[6], v[7]);
        }
        __syncthreads();
        const int wc = w * 16 + m16;  // this lane's column of the slab
        if constexpr (OUT) {
            // P = tril(xi kap^T) . D . b: the wavefront's row tile
            for (int rt = w; rt < NT; rt += 4)
                for (int ct = 0; ct <= rt; ++ct) {
                    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                    for (int k = 0; k < DKP; k += 16) {
                        const float4 xa = *reinterpret_cast<const float4*>(&Xi[(rt * 16 + m16) * LK + k + 4 * g4]);
                        const float4 kb = *reinterpret_cast<const float4*>(&Ka[(ct * 16 + m16) * LK + k + 4 * g4]);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.x, kb.x, acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.y, kb.y, acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.z, kb.z, acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.w, kb.w, acc, 0, 0, 0);
                    }
                    float f = dc.in[ct * 16 + m16];
                    if (ct < rt) {
                        f *= dc.suf[ct * 16 + m16];
                        for (int b = ct + 1; b < rt; ++b) f *= dc.tot[b];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = 4 * g4 + i;
                        const float d = ct == rt ? dc.diag[rt][t][m16] : dc.pre[rt * 16 + t];
                        // the masked half is zero whatever its product is (NaN or infinity among later tokens)
                        P[(rt * 16 + t) * LP + ct * 16 + m16] = ct == rt && t < m16 ? 0.f : acc[i] * (d * f);
                    }
                }
            __syncthreads();
#pragma unroll 1
            for (int rt = 0; rt < NT; ++rt) {
                f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < DKT; ++k) {
                    const float4 xa = *reinterpret_cast<const float4*>(&Xi[(rt * 16 + m16) * LK + k * 16 + 4 * g4]);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.x, X[k][0], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.y, X[k][1], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.z, X[k][2], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(xa.w, X[k][3], acc, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] *= dc.before(rt * 16 + 4 * g4 + i);
                for (int ct = 0; ct <= rt; ++ct) {
                    const float4 p = *reinterpret_cast<const float4*>(&P[(rt * 16 + m16) * LP + ct * 16 + 4 * g4]);
                    const float* om = &Om[(ct * 16 + 4 * g4) * LV + wc];
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p.x, om[0], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p.y, om[LV], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p.z, om[2 * LV], acc, 0, 0, 0);
                    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(p.w, om[3 * LV], acc, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = rt * 16 + 4 * g4 + i;
                    const bool ok = j < n && col_ok;
                    const int64_t t = row0 + (j < n ? token(j) : lo);
                    if (a.dot) {  // the row's product with `with`, over this slab's columns
                        float d = ok ? acc[i] * load1(a.with, a.with_bf16, t * a.DV + col) : 0.f;
                        for (int m = 1; m < 16; m <<= 1) d += __shfl_xor(d, m);
                        if (m16 == 0) dots[w][j] = d;
                    }
                    if (ok) a.out[t * a.DV + col] = a.o ? acc[i] * a.o[t] : acc[i];
                }
            }
            if (a.dot) {
                __syncthreads();
                if (tid < n)
                    a.dot[((int64_t)slab * a.NS + s) * a.T + token(tid)] = (dots[0][tid] + dots[1][tid]) + (dots[2][tid] + dots[3][tid]);
            }
        }
        const float total = dc.total();
        segdec *= total;
#pragma unroll
        for (int k = 0; k < DKT; ++k) X[k] *= total;
#pragma unroll 1
        for (int st = 0; st < NT; ++st) {
            float om[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = st * 16 + 4 * g4 + i;
                om[i] = Om[j * LV + wc] * (dc.after(j) * dc.in[j]);
            }
#pragma unroll
            for (int k = 0; k < DKT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    X[k] = __builtin_amdgcn_mfma_f32_16x16x4f32(Ka[(st * 16 + 4 * g4 + i) * LK + k * 16 + m16], om[i], X[k], 0, 0, 0);
        }
    }
    if (a.Xend) {
        const int64_t base = OUT ? s * (int64_t)a.DK * a.DV : st0;
#pragma unroll
        for (int k = 0; k < DKT; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = k * 16 + 4 * g4 + i;
                if (r < a.DK && col_ok) a.Xend[base + r * (int64_t)a.DV + col] = X[k][i];
            }
    }
    if (!OUT && slab == 0 && tid == 0) a.segdec[seg * a.NS + s] = segdec;
}

// The segments' own sums -> their starting states, and the state after the last
// one. Backwards, the segments run from the last, and the end is what flows
// into the state before token 0 (decayed by its gate).
__global__ __launch_bounds__(256) void dense_carry_kernel(CarryArgs a) {
    const int64_t per = a.per, i4 = ((int64_t)blockIdx.x * 256 + threadIdx.x);
    if (i4 >= a.NS * per / 4) return;
    const int64_t s = i4 / (per / 4), e = i4 % (per / 4);
    float4 X = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.X0) X = reinterpret_cast<const float4*>(a.X0)[i4];
    for (int j = 0; j < a.nseg; ++j) {
        const int seg = a.rev ? a.nseg - 1 - j : j;
        float4* p = reinterpret_cast<float4*>(a.ws) + (seg * a.NS + s) * (per / 4) + e;
        const float4 own = *p;
        const float d = a.segdec[seg * a.NS + s];
        *p = X;
        X = make_float4(fmaf(d, X.x, own.x), fmaf(d, X.y, own.y), fmaf(d, X.z, own.z), fmaf(d, X.w, own.w));
    }
    if (a.Xend) {
        const float d = a.rev && a.T > 0 ? a.gate[s * a.T] : 1.f;
        reinterpret_cast<float4*>(a.Xend)[i4] = make_float4(d * X.x, d * X.y, d * X.z, d * X.w);
    }
}

// Gates' gradients: a workgroup per (stream, segment). The segment's end value
// <alpha_{t+1} G_{t+1}, S_t>, then the running sum back over its tokens.
__global__ __launch_bounds__(256) void dense_gates_kernel(DenseGatesArgs a) {
    __shared__ float part[4];
    __shared__ float run[4];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int seg = (int)(blockIdx.x % a.nseg);
    const int64_t s = blockIdx.x / a.nseg;
    const int64_t lo = (int64_t)seg * a.L, hi = lo + a.L < a.T ? lo + a.L : a.T;
    const bool last = seg + 1 == a.nseg;
    float carry = 0.f;
    if (!last || a.has_dS) {
        const float4* G = reinterpret_cast<const float4*>(a.G + (seg * a.NS + s) * a.per);
        const float4* S = reinterpret_cast<const float4*>(last ? a.ST + s * a.per : a.S + ((seg + 1) * a.NS + s) * a.per);
        float d = 0.f;
        for (int64_t e = tid; e < a.per / 4; e += 256) {
            const float4 g = G[e], x = S[e];
            d = fmaf(g.x, x.x, fmaf(g.y, x.y, fmaf(g.z, x.z, fmaf(g.w, x.w, d))));
        }
        for (int m = 1; m < 64; m <<= 1) d += __shfl_xor(d, m);
        if (lane == 0) part[w] = d;
        __syncthreads();
        carry = ((part[0] + part[1]) + (part[2] + part[3])) * (last ? 1.f : a.alpha[s * a.T + hi]);
    }
    for (int64_t e = hi; e > lo; e -= 256) {  // 256 tokens from the end; this thread's is e - 1 - tid
        const int64_t t = e - 1 - tid;
        float x = 0.f;
        if (t >= lo) {
            float qdq = 0.f, db = 0.f;
            for (int p = 0; p < a.nslab_q; ++p) qdq += a.qdq[((int64_t)p * a.NS + s) * a.T + t];
            for (int p = 0; p < a.nslab_k; ++p) db += a.kdk[((int64_t)p * a.NS + s) * a.T + t];
            a.dbeta[s * a.T + t] = db;
            x = qdq - a.beta[s * a.T + t] * db;
        }
        for (int m = 1; m < 64; m <<= 1) {
            const float y = __shfl_up(x, m);
            if (lane >= m) x += y;
        }
        __syncthreads();
        if (lane == 63) run[w] = x;
        __syncthreads();
        for (int b = 0; b < w; ++b) x += run[b];
        if (t >= lo) a.dlog_alpha[s * a.T + t] = carry + x;
        carry += (run[0] + run[1]) + (run[2] + run[3]);
    }
}

// A few tokens a call (decoding): the state is read and written once, as rows
// of 64 columns; thread (r, c) holds rows r + 16 i, columns 4c .. 4c + 3.
template <int NR>
__global__ __launch_bounds__(256) void dense_step_kernel(DenseArgs a) {
    __shared__ float red[16][DENSE_SLAB];
    const int tid = threadIdx.x, r = tid >> 4, c = tid & 15;
    const int slab = (int)(blockIdx.x % a.nslab);
    const int64_t s = blockIdx.x / a.nslab;
    const int col = slab * DENSE_SLAB + 4 * c;
    const bool col_ok = col < a.DV;
    const int64_t st = s * (int64_t)a.DK * a.DV + col;
    float4 X[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        X[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.X0 && col_ok && r + 16 * i < a.DK) X[i] = *reinterpret_cast<const float4*>(a.X0 + st + (int64_t)(r + 16 * i) * a.DV);
    }
    for (int64_t t = s * a.T; t < (s + 1) * a.T; ++t) {
        const float g = a.a[t], b = a.b[t];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), y = v;
        if (col_ok) {
            if (a.omg_bf16) {
                const uint2 p = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.omg) + t * a.DV + col);
                v = make_float4(b * bf_lo(p.x), b * bf_hi(p.x), b * bf_lo(p.y), b * bf_hi(p.y));
            } else {
                const float4 p = *reinterpret_cast<const float4*>(static_cast<const float*>(a.omg) + t * a.DV + col);
                v = make_float4(b * p.x, b * p.y, b * p.z, b * p.w);
            }
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (r + 16 * i >= a.DK) break;
            const float k = load1(a.kap, a.kap_bf16, t * a.DK + r + 16 * i);
            const float q = load1(a.xi, a.xi_bf16, t * a.DK + r + 16 * i);
            X[i] = make_float4(fmaf(g, X[i].x, k * v.x), fmaf(g, X[i].y, k * v.y), fmaf(g, X[i].z, k * v.z), fmaf(g, X[i].w, k * v.w));
            y = make_float4(fmaf(q, X[i].x, y.x), fmaf(q, X[i].y, y.y), fmaf(q, X[i].z, y.z), fmaf(q, X[i].w, y.w));
        }
        __syncthreads();
        *reinterpret_cast<float4*>(&red[r][4 * c]) = y;
        __syncthreads();
        if (tid < DENSE_SLAB && slab * DENSE_SLAB + tid < a.DV) {
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) o += red[i][tid];
            a.out[t * a.DV + slab * DENSE_SLAB + tid] = o;
        }
    }
    if (a.Xend && col_ok)
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (r + 16 * i < a.DK) *reinterpret_cast<float4*>(a.Xend + st + (int64_t)(r + 16 * i) * a.DV) = X[i];
}

template <int DKT, int C, bool OUT>
hipError_t launch_dense_t(const DenseArgs& a, hipStream_t st) {
    constexpr int DKP = DKT * 16;
    constexpr int bytes = 4 * (C * (DKP + 4) * (OUT ? 2 : 1) + C * (DENSE_SLAB + 4) + (OUT ? C * (C + 4) : 0));
    static_assert(bytes + sizeof(Decay<C>) + 4 * C * 4 <= 160 * 1024, "a workgroup's LDS");
    hipLaunchKernelGGL((dense_kernel<DKT, C, OUT>), dim3((unsigned)(a.NS * a.nseg * a.nslab)), dim3(256), bytes, st, a);
    return hipGetLastError();
}

template <bool OUT>
hipError_t launch_dense(DenseArgs a, hipStream_t st) {
    a.nslab = (a.DV + DENSE_SLAB - 1) / DENSE_SLAB;
    if (a.DK <= 64) return launch_dense_t<4, 64, OUT>(a, st);
    if (a.DK <= 128) return launch_dense_t<8, 64, OUT>(a, st);
    return launch_dense_t<16, 32, OUT>(a, st);
}

hipError_t launch_carry(const CarryArgs& a, hipStream_t st) {
    const int64_t n = a.NS * a.per / 4;
    hipLaunchKernelGGL(dense_carry_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
    return hipGetLastError();
}

// Tokens of one call up to which the state is walked token by token.
constexpr int64_t STEP_TOKENS = 8;

// Segment length: enough workgroups for two per CU, segments of at least 256
// tokens (a segment costs two passes over a state), a multiple of the chunk.
int64_t segment_len(int64_t NS, int64_t T, int dv, int64_t most) {
    const int64_t slabs = (dv + DENSE_SLAB - 1) / DENSE_SLAB;
    int64_t want = (512 + NS * slabs - 1) / (NS * slabs);
    int64_t L = (T + want - 1) / want;
    if (L < 256) L = 256;
    if (L > most) L = most;
    return (L + 63) / 64 * 64;
}

struct DenseLayout {
    int64_t L, nseg, states, decs, bytes;
};
DenseLayout forward_layout(int64_t NS, int64_t T, int dk, int dv) {
    DenseLayout y{};
    y.L = segment_len(NS, T, dv, T);
    y.nseg = (T + y.L - 1) / y.L;
    if (T <= STEP_TOKENS || y.nseg == 1) return DenseLayout{y.L, 1, 0, 0, 0};
    y.states = y.nseg * NS * (int64_t)dk * dv * 4;
    y.decs = (y.nseg * NS * 4 + 255) / 256 * 256;
    y.bytes = y.states + y.decs;
    return y;
}
// the running sums of the gates' gradients take at most this many tokens
constexpr int64_t BWD_SEGMENT = 512;
struct DenseBwdLayout {
    int64_t L, nseg, states, one, decs, dq, dk, bytes;
};
DenseBwdLayout backward_layout(int64_t NS, int64_t T, int dk, int dv) {
    DenseBwdLayout y{};
    y.L = segment_len(NS, T, dv, BWD_SEGMENT);
    y.nseg = (T + y.L - 1) / y.L;
    y.one = (NS * (int64_t)dk * dv * 4 + 255) / 256 * 256;
    y.states = (y.nseg * NS * (int64_t)dk * dv * 4 + 255) / 256 * 256;
    y.decs = (y.nseg * NS * 4 + 255) / 256 * 256;
    const int64_t slabs = (dk + DENSE_SLAB - 1) / DENSE_SLAB;
    y.dq = (slabs * NS * T * 4 + 255) / 256 * 256;
    y.dk = y.dq;
    y.bytes = 2 * y.states + y.one + y.decs + y.dq + y.dk;
    return y;
}

}  // namespace

int64_t dense_workspace_bytes(int64_t NS, int64_t T, int dk, int dv) { return forward_layout(NS, T, dk, dv).bytes; }
int64_t dense_backward_workspace_bytes(int64_t NS, int64_t T, int dk, int dv) {
    return backward_layout(NS, T, dk, dv).bytes;
}

hipError_t launch_dense_forward(const DenseFwdArgs& f, hipStream_t st) {
    const DenseLayout y = forward_layout(f.NS, f.T, f.dk, f.dv);
    DenseArgs a{};
    a.xi = f.q; a.kap = f.k; a.omg = f.v;
    a.xi_bf16 = a.kap_bf16 = a.omg_bf16 = f.bf16;
    a.a = f.alpha; a.b = f.beta; a.out = f.y;
    a.NS = f.NS; a.T = f.T; a.L = y.L; a.nseg = (int)y.nseg;
    a.DK = f.dk; a.DV = f.dv;
    a.X0 = f.S0; a.x_row = f.dv; a.x_col = 1;
    a.Xend = f.S;
    if (f.T <= STEP_TOKENS) {
        a.nslab = (a.DV + DENSE_SLAB - 1) / DENSE_SLAB;
        const dim3 grid((unsigned)(a.NS * a.nslab));
        if (a.DK <= 64) hipLaunchKernelGGL(dense_step_kernel<4>, grid, dim3(256), 0, st, a);
        else if (a.DK <= 128) hipLaunchKernelGGL(dense_step_kernel<8>, grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL(dense_step_kernel<16>, grid, dim3(256), 0, st, a);
        return hipGetLastError();
    }
    if (y.nseg == 1) return launch_dense<true>(a, st);
    char* ws = static_cast<char*>(f.workspace);
    float* states = reinterpret_cast<float*>(ws);
    float* decs = reinterpret_cast<float*>(ws + y.states);
    DenseArgs p = a;
    p.X0 = nullptr; p.Xend = states; p.segdec = decs;
    hipError_t e = launch_dense<false>(p, st);
    if (e != hipSuccess) return e;
    CarryArgs c{};
    c.ws = states; c.segdec = decs; c.X0 = f.S0; c.Xend = f.S;
    c.NS = f.NS; c.per = (int64_t)f.dk * f.dv; c.nseg = (int)y.nseg;
    if ((e = launch_carry(c, st)) != hipSuccess) return e;
    a.X0 = states; a.X0_seg = true; a.Xend = nullptr;
    return launch_dense<true>(a, st);
}

hipError_t launch_dense_pass_on(const float* X0, float* X, int64_t NS, int64_t per, hipStream_t st) {
    CarryArgs c{};
    c.X0 = X0; c.Xend = X; c.NS = NS; c.per = per;
    return launch_carry(c, st);
}

hipError_t launch_dense_backward(const DenseBwdArgs& f, hipStream_t st) {
    const DenseBwdLayout y = backward_layout(f.NS, f.T, f.dk, f.dv);
    char* ws = static_cast<char*>(f.workspace);
    float* S = reinterpret_cast<float*>(ws);
    float* G = reinterpret_cast<float*>(ws + y.states);
    float* ST = reinterpret_cast<float*>(ws + 2 * y.states);
    float* decs = reinterpret_cast<float*>(ws + 2 * y.states + y.one);
    float* qdq = reinterpret_cast<float*>(ws + 2 * y.states + y.one + y.decs);
    float* kdk = reinterpret_cast<float*>(ws + 2 * y.states + y.one + y.decs + y.dq);
    const int64_t per = (int64_t)f.dk * f.dv;
    hipError_t e;
    DenseArgs base{};
    base.a = f.alpha; base.NS = f.NS; base.T = f.T; base.L = y.L; base.nseg = (int)y.nseg;
    CarryArgs c{};
    c.segdec = decs; c.NS = f.NS; c.per = per; c.nseg = (int)y.nseg; c.T = f.T; c.gate = f.alpha;

    DenseArgs p = base;  // S at the segments' starts, and after the last
    p.kap = f.k; p.omg = f.v; p.kap_bf16 = p.omg_bf16 = f.bf16; p.b = f.beta;
    p.DK = f.dk; p.DV = f.dv; p.Xend = S; p.segdec = decs;
    if ((e = launch_dense<false>(p, st)) != hipSuccess) return e;
    c.ws = S; c.X0 = f.S0; c.Xend = ST;
    if ((e = launch_carry(c, st)) != hipSuccess) return e;

    p = base;            // G at the segments' ends, and what flows into S0
    p.kap = f.q; p.kap_bf16 = f.bf16; p.omg = f.dy; p.rev = true;
    p.DK = f.dk; p.DV = f.dv; p.Xend = G; p.segdec = decs;
    if ((e = launch_dense<false>(p, st)) != hipSuccess) return e;
    c.ws = G; c.X0 = f.dS; c.Xend = f.dS0; c.rev = true;
    if ((e = launch_carry(c, st)) != hipSuccess) return e;

    p = base;            // dq, and q . dq
    p.xi = f.dy; p.kap = f.v; p.kap_bf16 = f.bf16; p.omg = f.k; p.omg_bf16 = f.bf16; p.b = f.beta;
    p.DK = f.dv; p.DV = f.dk; p.X0 = S; p.X0_seg = true; p.x_row = 1; p.x_col = f.dv;
    p.out = f.dq; p.dot = qdq; p.with = f.q; p.with_bf16 = f.bf16;
    if ((e = launch_dense<true>(p, st)) != hipSuccess) return e;

    p = base;            // dk, and k . dk / beta
    p.xi = f.v; p.xi_bf16 = f.bf16; p.kap = f.dy; p.omg = f.q; p.omg_bf16 = f.bf16; p.o = f.beta; p.rev = true;
    p.DK = f.dv; p.DV = f.dk; p.X0 = G; p.X0_seg = true; p.x_row = 1; p.x_col = f.dv;
    p.out = f.dk_out; p.dot = kdk; p.with = f.k; p.with_bf16 = f.bf16;
    if ((e = launch_dense<true>(p, st)) != hipSuccess) return e;

    p = base;            // dv
    p.xi = f.k; p.xi_bf16 = f.bf16; p.kap = f.q; p.kap_bf16 = f.bf16; p.omg = f.dy; p.o = f.beta; p.rev = true;
    p.DK = f.dk; p.DV = f.dv; p.X0 = G; p.X0_seg = true; p.x_row = f.dv; p.x_col = 1;
    p.out = f.dv_out;
    if ((e = launch_dense<true>(p, st)) != hipSuccess) return e;

    DenseGatesArgs g{};
    g.G = G; g.S = S; g.ST = ST; g.qdq = qdq; g.kdk = kdk; g.alpha = f.alpha; g.beta = f.beta;
    g.dlog_alpha = f.dlog_alpha; g.dbeta = f.dbeta; g.has_dS = f.dS != nullptr;
    g.NS = f.NS; g.T = f.T; g.L = y.L; g.per = per; g.nseg = (int)y.nseg;
    g.nslab_q = g.nslab_k = (f.dk + DENSE_SLAB - 1) / DENSE_SLAB;
    hipLaunchKernelGGL(dense_gates_kernel, dim3((unsigned)(f.NS * y.nseg)), dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace sdm
