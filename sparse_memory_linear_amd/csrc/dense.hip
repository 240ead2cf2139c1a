// dense.hip -- the dense gated recurrence on gfx950: a d_k x d_v state per head
// in which every token decays all rows and adds one outer product,
//   S_t = alpha_t S_{t-1} + beta_t k_t (x) v_t,     y_t = q_t S_t,
// and its gradients: linear attention with a forget and an input gate, the same gates,
// v and y as the sparse scan's. (Its rule adds beta k (x) v as it is; the scan's takes
// off what the rows hold before it adds, and nothing here normalises the read.)
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
// Segments: with few streams the tokens are split into segments; a pass leaves
// each segment's own sum, a second adds them up over the segments (giving each
// one's starting state), and the last computes the outputs. The backward does so
// for S and G in one launch, and for dq, dk and dv in one.
//
// Measured at 4 x 8 streams, T = 8192, 128 x 128, bf16 rows (32 streams, 16
// segments of 512 tokens each): forward 141 us in all (segments' sums 36, carry 14, y 84;
// 342 MB that it cannot do without: 72 us at a copy's 4.75 TB/s), backward 494 us (sums 97,
// carry 23, gradients 358, gates 22; 749 MB, 158 us). The forward moves 604 MB, k and v twice
// and the states four times: the sums 168 MB at 4.6 TB/s, the carry 67 at 4.9, y 369 at 4.4,
// where the vector units are busy for half of the time too (dense_pass.h). The gradients are
// bound by vector and matrix instructions. With few streams the carry is a chain of loads: 0.4 us
// a segment.
#include "dense_pass.h"

namespace sdm {

namespace {

// the running sums of the gates' gradients start anew at segments of at most this many tokens
constexpr int64_t BWD_SEGMENT = 512;
constexpr int STEP_COLS = 64;  // columns of X a workgroup of the one-token form

// The segments' own sums -> their starting states, and the state after the last
// one. Backwards, the segments run from the last, and the end is what flows
// into the state before token 0 (decayed by its gate).
__global__ __launch_bounds__(256) void dense_carry_kernel(CarryArgs s0, CarryArgs s1) {
    const CarryArgs& a = blockIdx.y ? s1 : s0;
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

// Gates' gradients: a workgroup per (stream, segment), a row of 32 lanes a chunk, its last
// token in lane 0. With e the value of <alpha_{t+1} G_{t+1}, S_t> at a chunk's end: at the
// segment's end it is that product of the two states; over a chunk it changes by what the two
// passes found to flow into and out of the chunk, and within one E_t = e + the sum over u >= t
// of q_u . dq_u - k_u . dk_u. So a rounding reaches no further than a chunk, but for the chunks'
// own sums, which hold only what crosses their bounds. Nothing passes a gate of 0: E is exactly
// 0 there and the sums begin anew, so that a sequence's rounding stays out of the one before it.
__global__ __launch_bounds__(256) void dense_gates_kernel(DenseGatesArgs a) {
    constexpr int C = DENSE_CHUNK, NI = BWD_SEGMENT / 256;
    static_assert(C == 32 && BWD_SEGMENT % 256 == 0, "a chunk is half a wavefront");
    __shared__ float part[4];
    __shared__ float diff[BWD_SEGMENT / C], at_end[BWD_SEGMENT / C];
    __shared__ bool anew[BWD_SEGMENT / C];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, in = tid & (C - 1);
    const int seg = (int)(blockIdx.x % a.nseg);
    const int64_t s = blockIdx.x / a.nseg;
    const int64_t lo = (int64_t)seg * a.L, hi = lo + a.L < a.T ? lo + a.L : a.T;
    const bool last = seg + 1 == a.nseg;
    const int nch = (int)((hi - lo + C - 1) / C);
    float d = 0.f;
    if (!last || a.has_dS) {
        const float4* G = reinterpret_cast<const float4*>(a.G + (seg * a.NS + s) * a.per);
        const float4* S = reinterpret_cast<const float4*>(last ? a.ST + s * a.per : a.S + ((seg + 1) * a.NS + s) * a.per);
#pragma unroll 8
        for (int e = tid; e < (int)(a.per / 4); e += 256) d += dot4(G[e], S[e]);
        d *= last ? 1.f : a.alpha[s * a.T + hi];
    }
    d = wave_sum(d);
    if (lane == 0) part[w] = d;
    float x[NI];
    int shut[NI];  // a gate of 0 at this token or behind it in the chunk
    int64_t t[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int c = (i * 256 + tid) / C;
        const int64_t c0 = lo + (int64_t)c * C, c1 = c0 + C < hi ? c0 + C : hi;
        t[i] = c1 - 1 - in;
        x[i] = 0.f;
        shut[i] = 0;
        if (c >= nch || t[i] < c0) {
            t[i] = -1;
        } else {
            float qdq = 0.f, db = 0.f;
            for (int p = 0; p < a.nslab; ++p) {
                qdq += a.qdq[(p * a.NS + s) * a.T + t[i]];
                db += a.kdk[(p * a.NS + s) * a.T + t[i]];
            }
            a.dbeta[s * a.T + t[i]] = db;
            shut[i] = a.alpha[s * a.T + t[i]] == 0.f;
            x[i] = shut[i] ? 0.f : qdq - a.beta[s * a.T + t[i]] * db;
        }
        for (int m = 1; m < C; m <<= 1) {
            const float y = __shfl_up(x[i], m, C);
            const int z = __shfl_up(shut[i], m, C);
            if (in >= m) {
                if (!shut[i]) x[i] += y;
                shut[i] |= z;
            }
        }
        if (c < nch && t[i] == c0) {  // over the chunk
            float v = x[i];
            if (!shut[i]) {
                v = 0.f;
                for (int p = 0; p < a.nslab; ++p) {
                    const int64_t at = (p * a.NS + s) * a.nchunk + c0 / C;
                    v += a.inter_q[at] - a.inter_k[at];
                }
            }
            diff[c] = v;
            anew[c] = shut[i] != 0;
        }
    }
    __syncthreads();
    if (tid == 0) {
        float e = (part[0] + part[1]) + (part[2] + part[3]);
        for (int c = nch - 1; c >= 0; --c) {
            at_end[c] = e;
            e = anew[c] ? diff[c] : e + diff[c];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (t[i] >= 0) a.dlog_alpha[s * a.T + t[i]] = shut[i] ? x[i] : at_end[(i * 256 + tid) / C] + x[i];
}

__device__ __forceinline__ float load1(const void* p, bool bf16, int64_t e) {
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[e] << 16) : static_cast<const float*>(p)[e];
}

// One token (decoding): the state is read and written once, as rows of 64
// columns; thread (r, c) takes rows r + 16 i, columns 4c .. 4c + 3. HBM-bound: 2048
// states of 128 x 128 in 62.6 us over three sets in turn, 4.3 TB/s (41.5 over one, part of
// which stays in the memory-side cache). The chunked pass takes 62.6 (50.9) for one token and 62.9
// for two there, but 31 us against 23 for 4096 states of 64 x 64, and 195 against 112 for
// 4096 of 128 x 128 with fp32 rows.
template <int NR>
__global__ __launch_bounds__(256) void dense_step_kernel(DenseFwdArgs a) {
    __shared__ float red[16][STEP_COLS];
    const int tid = threadIdx.x, r = tid >> 4, c = tid & 15;
    const int nslab = (a.dv + STEP_COLS - 1) / STEP_COLS, slab = (int)(blockIdx.x % nslab);
    const int64_t s = blockIdx.x / nslab;
    const int col = slab * STEP_COLS + 4 * c;
    const bool col_ok = col < a.dv;
    const int64_t st = s * (int64_t)a.dk * a.dv + col;
    const float g = a.alpha[s], b = a.beta[s];
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), y = v;
    if (col_ok) {
        if (a.bf16) {
            const uint2 p = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.v) + s * a.dv + col);
            v = make_float4(b * bf_lo(p.x), b * bf_hi(p.x), b * bf_lo(p.y), b * bf_hi(p.y));
        } else {
            v = f4_scale(b, *reinterpret_cast<const float4*>(static_cast<const float*>(a.v) + s * a.dv + col));
        }
    }
    float4 X[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        X[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.S0 && col_ok && r + 16 * i < a.dk) X[i] = *reinterpret_cast<const float4*>(a.S0 + st + (int64_t)(r + 16 * i) * a.dv);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = r + 16 * i;
        if (row >= a.dk) break;
        const float k = load1(a.k, a.bf16, s * a.dk + row), q = load1(a.q, a.bf16, s * a.dk + row);
        X[i] = make_float4(fmaf(g, X[i].x, k * v.x), fmaf(g, X[i].y, k * v.y), fmaf(g, X[i].z, k * v.z), fmaf(g, X[i].w, k * v.w));
        y = f4_fma(q, X[i], y);
        if (a.S && col_ok) *reinterpret_cast<float4*>(a.S + st + (int64_t)row * a.dv) = X[i];
    }
    *reinterpret_cast<float4*>(&red[r][4 * c]) = y;
    __syncthreads();
    if (tid < STEP_COLS && slab * STEP_COLS + tid < a.dv) {
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) o += red[i][tid];
        a.y[s * a.dv + slab * STEP_COLS + tid] = o;
    }
}

// b: another set of the same sizes in the same launch, or nullptr
hipError_t launch_carry(const CarryArgs& a, const CarryArgs* b, hipStream_t st) {
    const int64_t n = a.NS * a.per / 4;
    hipLaunchKernelGGL(dense_carry_kernel, dim3((unsigned)((n + 255) / 256), b ? 2 : 1), dim3(256), 0, st, a, b ? *b : a);
    return hipGetLastError();
}

// Segment length: enough workgroups for two per CU (a state per segment and
// stream, so some 512 of them whatever the length), of at least two chunks.
int64_t segment_len(int64_t NS, int64_t T, int dv, int64_t most) {
    const int64_t slabs = (dv + dense_slab(dv) - 1) / dense_slab(dv);
    const int64_t want = (512 + NS * slabs - 1) / (NS * slabs);
    int64_t L = (T + want - 1) / want;
    if (L > most) L = most;
    if (L < 2 * DENSE_CHUNK) L = 2 * DENSE_CHUNK;
    return (L + DENSE_CHUNK - 1) / DENSE_CHUNK * DENSE_CHUNK;
}

struct DenseLayout {
    int64_t L, nseg, states, decs, bytes;
};
DenseLayout forward_layout(int64_t NS, int64_t T, int dk, int dv) {
    DenseLayout y{};
    y.L = segment_len(NS, T, dv, T);
    y.nseg = (T + y.L - 1) / y.L;
    // One segment a stream (one launch) unless segments are quicker. In us: a chunk takes 2.5, in the
    // first pass some 0.6 of that; two more launches 6; a segment's state is moved four times at 4.75
    // TB/s. (Measured, one / segments: 8 streams of 128 x 128, T = 128: 17 / 21, 256: 27 / 21; 64 streams,
    // 384: 39 / 38, 1024: 91 / 56; of 256 x 256, 512: 71 / 101, 1024: 134 / 152; 256 streams of 64 x 64, 512:
    // 29 / 37, 1024: 52 / 61. The chunk's time is that of bf16 rows and 128 x 128; with fp32 rows the same
    // are 26 / 26, 46 / 27; 68 / 55, 178 / 99; 141 / 154, 270 / 253; 45 / 58, 84 / 102.)
    const double one = 2.5 * T / DENSE_CHUNK;
    const double many = 4.0 * y.L / DENSE_CHUNK + 6 + 16e-6 * y.nseg * NS * dk * dv / 4.75;
    if (y.nseg == 1 || one <= many) return DenseLayout{T, 1, 0, 0, 0};
    y.states = y.nseg * NS * (int64_t)dk * dv * 4;
    y.decs = (y.nseg * NS * 4 + 255) / 256 * 256;
    y.bytes = y.states + y.decs;
    return y;
}
struct DenseBwdLayout {
    int64_t L, nseg, states, one, decs, dots, nchunk, inter, bytes;
    int slabs;
};
DenseBwdLayout backward_layout(int64_t NS, int64_t T, int dk, int dv) {
    DenseBwdLayout y{};
    y.L = segment_len(NS, T, dv, BWD_SEGMENT);
    y.nseg = (T + y.L - 1) / y.L;
    y.one = (NS * (int64_t)dk * dv * 4 + 255) / 256 * 256;
    y.states = (y.nseg * NS * (int64_t)dk * dv * 4 + 255) / 256 * 256;
    y.decs = (y.nseg * NS * 4 + 255) / 256 * 256;
    y.slabs = (dk + dense_slab(dk) - 1) / dense_slab(dk);
    y.dots = (y.slabs * NS * T * 4 + 255) / 256 * 256;
    y.nchunk = (T + DENSE_CHUNK - 1) / DENSE_CHUNK;
    y.inter = (y.slabs * NS * y.nchunk * 4 + 255) / 256 * 256;
    y.bytes = 2 * y.states + y.one + 2 * y.decs + 2 * y.dots + 2 * y.inter;
    return y;
}

}  // namespace

int64_t dense_workspace_bytes(int64_t NS, int64_t T, int dk, int dv) { return forward_layout(NS, T, dk, dv).bytes; }
int64_t dense_backward_workspace_bytes(int64_t NS, int64_t T, int dk, int dv) {
    return backward_layout(NS, T, dk, dv).bytes;
}

hipError_t launch_dense_forward(const DenseFwdArgs& f, hipStream_t st) {
    const DenseLayout y = forward_layout(f.NS, f.T, f.dk, f.dv);
    if (f.T == 1) {
        const dim3 grid((unsigned)(f.NS * ((f.dv + STEP_COLS - 1) / STEP_COLS)));
        if (f.dk <= 64) hipLaunchKernelGGL(dense_step_kernel<4>, grid, dim3(256), 0, st, f);
        else if (f.dk <= 128) hipLaunchKernelGGL(dense_step_kernel<8>, grid, dim3(256), 0, st, f);
        else hipLaunchKernelGGL(dense_step_kernel<16>, grid, dim3(256), 0, st, f);
        return hipGetLastError();
    }
    DenseArgs a{};
    a.a = f.alpha; a.beta = f.beta;
    a.NS = f.NS; a.T = f.T; a.L = y.L; a.nseg = (int)y.nseg;
    a.DK = f.dk; a.DV = f.dv;
    a.kap = f.k; a.omg = f.v;
    if (y.nseg > 1) {
        char* ws = static_cast<char*>(f.workspace);
        float* states = reinterpret_cast<float*>(ws);
        DenseArgs p = a;
        p.Xend = states; p.segdec = reinterpret_cast<float*>(ws + y.states);
        hipError_t e = f.bf16 ? launch_dense_s(p, st) : launch_dense_s_f32(p, st);
        if (e != hipSuccess) return e;
        CarryArgs c{};
        c.ws = states; c.segdec = p.segdec; c.X0 = f.S0; c.Xend = f.S;
        c.NS = f.NS; c.per = (int64_t)f.dk * f.dv; c.nseg = (int)y.nseg;
        if ((e = launch_carry(c, nullptr, st)) != hipSuccess) return e;
        a.X0 = states;
    } else {
        a.X0 = f.S0; a.Xend = f.S;
    }
    a.xi = f.q; a.out = f.y;
    return f.bf16 ? launch_dense_y(a, st) : launch_dense_y_f32(a, st);
}

hipError_t launch_dense_pass_on(const float* X0, float* X, int64_t NS, int64_t per, hipStream_t st) {
    CarryArgs c{};
    c.X0 = X0; c.Xend = X; c.NS = NS; c.per = per;
    return launch_carry(c, nullptr, st);
}

hipError_t launch_dense_backward(const DenseBwdArgs& f, hipStream_t st) {
    const DenseBwdLayout y = backward_layout(f.NS, f.T, f.dk, f.dv);
    char* ws = static_cast<char*>(f.workspace);
    float* S = reinterpret_cast<float*>(ws);
    float* G = reinterpret_cast<float*>(ws + y.states);
    float* ST = reinterpret_cast<float*>(ws + 2 * y.states);
    float* decS = reinterpret_cast<float*>(ws + 2 * y.states + y.one);
    float* decG = reinterpret_cast<float*>(ws + 2 * y.states + y.one + y.decs);
    char* dots = ws + 2 * y.states + y.one + 2 * y.decs;
    float* qdq = reinterpret_cast<float*>(dots);
    float* kdk = reinterpret_cast<float*>(dots + y.dots);
    float* inter_q = reinterpret_cast<float*>(dots + 2 * y.dots);
    float* inter_k = reinterpret_cast<float*>(dots + 2 * y.dots + y.inter);
    const int64_t per = (int64_t)f.dk * f.dv;
    hipError_t e;
    DenseArgs base{};
    base.a = f.alpha; base.beta = f.beta; base.NS = f.NS; base.T = f.T; base.L = y.L; base.nseg = (int)y.nseg;
    // S at the segments' starts and after the last, G at their ends and what flows into S0
    DenseArgs ps = base, pg = base;
    ps.kap = f.k; ps.omg = f.v; ps.DK = f.dk; ps.DV = f.dv; ps.Xend = S; ps.segdec = decS;
    pg.kap = f.q; pg.omg = f.dy; pg.DK = f.dk; pg.DV = f.dv; pg.Xend = G; pg.segdec = decG;
    if ((e = f.bf16 ? launch_dense_sg(ps, pg, st) : launch_dense_sg_f32(ps, pg, st)) != hipSuccess) return e;
    CarryArgs cs{}, cg{};
    cs.ws = S; cs.segdec = decS; cs.X0 = f.S0; cs.Xend = ST;
    cs.NS = f.NS; cs.per = per; cs.nseg = (int)y.nseg; cs.T = f.T; cs.gate = f.alpha;
    cg = cs;
    cg.ws = G; cg.segdec = decG; cg.X0 = f.dS; cg.Xend = f.dS0; cg.rev = true;
    if ((e = launch_carry(cs, &cg, st)) != hipSuccess) return e;

    DenseArgs pq = base, pk = base, pv = base;
    pq.xi = f.dy; pq.kap = f.v; pq.omg = f.k; pq.DK = f.dv; pq.DV = f.dk; pq.X0 = S;  // dq, and q . dq
    pq.out = f.dq; pq.dot = qdq; pq.inter = inter_q; pq.with = f.q;
    pk.xi = f.v; pk.kap = f.dy; pk.omg = f.q; pk.DK = f.dv; pk.DV = f.dk; pk.X0 = G;  // dk, and k . dk / beta
    pk.out = f.dk_out; pk.dot = kdk; pk.inter = inter_k; pk.with = f.k;
    pv.xi = f.k; pv.kap = f.q; pv.omg = f.dy; pv.DK = f.dk; pv.DV = f.dv; pv.X0 = G;  // dv
    pv.out = f.dv_out;
    if ((e = f.bf16 ? launch_dense_grads(pq, pk, pv, st) : launch_dense_grads_f32(pq, pk, pv, st)) != hipSuccess) return e;

    DenseGatesArgs g{};
    g.G = G; g.S = S; g.ST = ST; g.qdq = qdq; g.kdk = kdk; g.alpha = f.alpha; g.beta = f.beta;
    g.dlog_alpha = f.dlog_alpha; g.dbeta = f.dbeta; g.has_dS = f.dS != nullptr;
    g.NS = f.NS; g.T = f.T; g.L = y.L; g.per = per; g.nseg = (int)y.nseg;
    g.inter_q = inter_q; g.inter_k = inter_k; g.nchunk = y.nchunk; g.nslab = y.slabs;
    hipLaunchKernelGGL(dense_gates_kernel, dim3((unsigned)(f.NS * y.nseg)), dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace sdm
