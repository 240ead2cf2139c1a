// dense_pass.h -- one pass of the dense gated recurrence (dense.hip says which
// recurrence and how its passes make the forward and the gradients).
//
//   X_u = a_u X_{u-1} + b_u kap_u (x) omg_u,    out_u = o_u xi_u X_u
//
// A workgroup carries SV = 16 NCT NW columns of X in registers over a segment's
// tokens, C = 32 at a time; a wavefront owns 16 NCT of them. Within a chunk, with
// D_ts = a_{s+1} .. a_t,
//   out = o (pre X_start + (tril(xi kap^T) . D . b) omg),   pre_t = a_c0 .. a_t
//   X_end = total X_start + sum_s kap_s (x) (D_end,s b_s omg_s).
// The decays are products of the gates, never quotients or differences of
// logarithms: a gate of 0 gives exact zeros and no 0/0. Off the diagonal blocks
// of 16 x 16, D_ts is the product from t's block start, the whole blocks
// between, and to s's block end; the diagonal block's wavefront forms its own.
//
// All four products run on bf16 matrix instructions (16x16x32, fp32 sums) with
// fp32 operands kept to fp32's precision: a value is cut into three bf16 planes
// of 8 bits each (high, middle, low; their sum is the value), and a product of an
// fp32 operand with a bf16 one takes 3 matrix products, of two fp32 operands 6.
// That is 1/3 and 1/6 of the bf16 rate, against 1/16 for the fp32 matrix instructions.
// The planes are rounded to nearest: a middle one is at most 2^-8 of the value and a low
// one 2^-17, so the terms left out (middle x low twice, low x low) are 2^-24 of the product
// or less, and of either sign. (Planes cut off would leave out up to 2^-21, always towards
// zero, for 1 to 4% less time: the forwards of 4x8x8192 x 128 x 128 142 us against 144, of
// 2x8x4096 x 256 x 256 139 against 145, all in bf16.)
//
// Layouts. xi and kap lie in LDS as rows (token-major, a plane an array), padded by
// 16 bytes so that 16 rows' pieces fall into different banks. A lane of the 16x16x32
// instruction takes 8 consecutive k; X's tiles are numbered so that the 8 rows that
// a lane's accumulators hold in tiles 2p and 2p+1 are 32p + 8 (lane / 16) + 0..7,
// so X goes from accumulator to operand without leaving its registers (a pass
// without outputs numbers them plainly, which spares the transposing reads bank conflicts). kap^T and omg as
// operands over the tokens come from the same rows by transposing LDS reads; their
// token order (4 (lane / 16) + i of two tiles of 16) is the accumulators', so P^T =
// kap xi^T is written by the wavefront that computes it in the order in which the
// others read it.
//
// What bounds it (4 x 8 streams, T = 8192, 128 x 128, bf16; per SIMD, in thousands of cycles):
// the y pass takes 173, of them 89 of vector instructions, 57 of matrix ones and, per CU, 49 of LDS,
// and moves its bytes at 4.4 TB/s; the three gradient passes 711, 354, 232 and 238. Nearly half of
// the vector instructions cut X into planes: with that left out (wrong results) y took 73 us in place of
// 87, with two of the three matrix products left out 93. Two planes would do with a relative error of
// 3e-6; three keep fp32's. Tried and dropped: chunks of 64 tokens (half the cutting, but spilled
// registers: 117 us against 90), fp32 matrix instructions (819 us for the forward against 287 for the
// first form of this one), residues of the planes by the bf16 dot instruction (its wait states cost what
// it saved: 92 us against 87).
#pragma once
#include <type_traits>

#include "sdm_buffer.h"
#include "sdm_internal.h"

namespace sdm {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// An element offset whose byte offset, in 2- and in 4-byte elements and give or take a
// chunk's rows, lies beyond every buffer (a buffer holds at most 64 KiB).
constexpr uint32_t FAR = 0x28000000u;

// two values' planes, packed: a's in the low half (the differences are exact, and leave 7
// bits for the last plane)
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& m, uint32_t& l) {
    h = RowFmt<true>::pk(a, b);
    a -= bf_lo(h); b -= bf_hi(h);
    m = RowFmt<true>::pk(a, b);
    l = __builtin_amdgcn_perm(__float_as_uint(b - bf_hi(m)), __float_as_uint(a - bf_lo(m)), 0x07060302u);
}
// 8 values -> three operand planes
__device__ __forceinline__ void split8(const float (&v)[8], uint4 (&p)[3]) {
    split2(v[0], v[1], p[0].x, p[1].x, p[2].x);
    split2(v[2], v[3], p[0].y, p[1].y, p[2].y);
    split2(v[4], v[5], p[0].z, p[1].z, p[2].z);
    split2(v[6], v[7], p[0].w, p[1].w, p[2].w);
}

// x times the values of the N lanes before (or behind) it in its row of 16; 1 beyond the row
template <int N>
__device__ __forceinline__ float times_before(float x) {
    return x * __int_as_float(__builtin_amdgcn_update_dpp(0x3F800000, __float_as_int(x), 0x110 + N, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ float times_behind(float x) {
    return x * __int_as_float(__builtin_amdgcn_update_dpp(0x3F800000, __float_as_int(x), 0x100 + N, 0xF, 0xF, false));
}
// products over the row's lanes up to and with this one, and from this one on
__device__ __forceinline__ float product_to(float x) {
    return times_before<8>(times_before<4>(times_before<2>(times_before<1>(x))));
}
__device__ __forceinline__ float product_from(float x) {
    return times_behind<8>(times_behind<4>(times_behind<2>(times_behind<1>(x))));
}

// acc += A B over the operands' planes
template <int NA, int NB>
__device__ __forceinline__ void mma(const uint4 (&a)[NA], const uint4 (&b)[NB], f32x4_t& acc) {
    auto one = [&](int i, int j) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a[i]), __builtin_bit_cast(bf16x8_t, b[j]),
                                                      acc, 0, 0, 0);
    };
#pragma unroll
    for (int s = 2; s >= 0; --s)  // the smallest terms first
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
                if (i + j == s) one(i, j);
}

// 8 elements from global memory: bf16 (one register quad) or fp32 (two)
template <int NP>
struct Piece;
template <>
struct Piece<1> {
    uint4 x;
    static constexpr uint32_t ESZ = 2;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
        const int4 v = ld_i4(r, off, 0);
        x = make_uint4((uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w);
    }
    __device__ __forceinline__ void store(char* lds, int) const { *reinterpret_cast<uint4*>(lds) = x; }
    __device__ __forceinline__ void store_raw(char* lds) const { *reinterpret_cast<uint4*>(lds) = x; }
};
template <>
struct Piece<3> {
    float4 x, y;
    static constexpr uint32_t ESZ = 4;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t off) {
        x = ld_f4(r, off, 0);
        y = ld_f4(r, off + 16u, 0);
    }
    __device__ __forceinline__ void store(char* lds, int plane) const {
        const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint4 p[3];
        split8(v, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint4*>(lds + i * plane) = p[i];
    }
    __device__ __forceinline__ void store_raw(char* lds) const {
        *reinterpret_cast<float4*>(lds) = x;
        *reinterpret_cast<float4*>(lds + 16) = y;
    }
};

// transposing read of 4 rows x 16 columns by 16 lanes: this lane's piece is 8
// bytes at p; it gets its own column of the 4 rows
__device__ __forceinline__ uint2 read_tr(const char* p) {
    typedef __attribute__((address_space(3))) s16x4_t lds_t;
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p));
}

// NX, NK, NO: planes of xi, kap and omg (1: bf16 in memory, 3: fp32).
// OUT: outputs (else only the segment's own state, from zero). REV: from the last
// token to the first, with a_u = alpha_{t+1}, b = 1, o = beta (else alpha_t, beta, 1).
// DOT: also the outputs' products with the rows `with`, and the starting states are
// taken transposed (the gradients over the value rows: dq and dk).
template <int DKT_, int NCT_, int NW_, int NX_, int NK_, int NO_, bool OUT_, bool REV_, bool DOT_>
struct DensePass {
    static constexpr int DKT = DKT_, NCT = NCT_, NW = NW_, C = DENSE_CHUNK, NX = NX_, NK = NK_, NO = NO_;
    static constexpr bool OUT = OUT_, REV = REV_, DOT = DOT_;
    static constexpr int WITH = NX == 3 && NK == 3 ? 4 : 2;          // bytes of `with`: q and k, as the other rows
    static constexpr int DKP = DKT * 16, SV = 16 * NCT * NW, NT = C / 16, THR = NW * 64;
    // bytes of an LDS row: rows read as operands are 16 apart of the banks' width, rows that
    // only transposing reads take (4 rows of 32 bytes at a time) 32
    static constexpr int RK = DKP * 2 + (OUT ? 16 : 32), RV = SV * 2 + 32;
    static constexpr int PK = C * RK, PV = C * RV;                   // bytes of a plane
    static constexpr int TILES = NT * (NT + 1) / 2;
    static constexpr int O_KA = 0, O_OM = O_KA + NK * PK, O_XI = O_OM + NO * PV, O_WI = O_XI + (OUT ? NX * PK : 0),
                         RW = SV * WITH + 32, ROWS = O_WI + (DOT ? C * RW : 0);
    // floats: two sets of a chunk's decays, outputs' products, their sums
    static constexpr int DEC = 4 * C + 2 * NT, FLOATS = 2 * DEC + (DOT ? 2 * NW * (C + 1) : 0);
    static constexpr int PBYTES = OUT ? TILES * 3 * 512 : 0;
    // the rows twice (the next chunk's are stored while this one's are read), unless that
    // keeps a second workgroup off the CU
    static constexpr int BUF = 2 * ROWS + PBYTES + FLOATS * 4 <= 80 * 1024 ? 2 : 1;
    static constexpr int O_P = BUF * ROWS, O_F = O_P + PBYTES, LDS = O_F + FLOATS * 4;
    static_assert(NT == 2, "tiles of P are numbered for 2 blocks");
    static_assert(LDS <= 160 * 1024, "a workgroup's LDS");
};

// One workgroup's pass: stream and segment us, column slab `slab`.
template <class P>
__device__ __forceinline__ void dense_pass(const DenseArgs& a, int64_t us, int slab, char* const lds) {
    constexpr int DKT = P::DKT, NCT = P::NCT, C = P::C, NT = P::NT, THR = P::THR, DKP = P::DKP, SV = P::SV, NW = P::NW;
    char* const Pf = lds + P::O_P;
    float* const dec = reinterpret_cast<float*>(lds + P::O_F);
    float* const dots = dec + 2 * P::DEC;  // [2][NW][C + 1]: per wavefront, the rows' products, and their part from X_start
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), m16 = lane & 15, g4 = lane >> 4;
    const int64_t s = us / a.nseg;  // stream
    const int seg = (int)(us % a.nseg);
    const int64_t lo = (int64_t)seg * a.L, hi = lo + a.L < a.T ? lo + a.L : a.T;
    const int c0 = slab * SV;
    const int64_t row0 = s * a.T, state = (seg * a.NS + s) * (int64_t)a.DK * a.DV;
    int col[NCT];
#pragma unroll
    for (int n = 0; n < NCT; ++n) col[n] = c0 + (w * NCT + n) * 16 + m16;

    // rows 32p + 8 g4 + 4h + i in X[2p + h][..][i]
    f32x4_t X[DKT][NCT];
#pragma unroll
    for (int k = 0; k < DKT; ++k)
#pragma unroll
        for (int n = 0; n < NCT; ++n) {
            X[k][n] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            const int r = 32 * (k >> 1) + 8 * g4 + 4 * (k & 1);
            if (P::OUT && a.X0 && r < a.DK && col[n] < a.DV) {  // DK a multiple of 8: 4 rows at once
                if (P::DOT) {
                    const float4 v = *reinterpret_cast<const float4*>(a.X0 + state + (int64_t)col[n] * a.DK + r);
                    X[k][n] = f32x4_t{v.x, v.y, v.z, v.w};
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) X[k][n][i] = a.X0[state + (int64_t)(r + i) * a.DV + col[n]];
                }
            }
        }

    constexpr int KP = (C * (DKP / 8) + THR - 1) / THR, VP = (C * (SV / 8) + THR - 1) / THR;  // pieces a thread
    Piece<P::NK> pk[KP];
    Piece<P::NX> px[P::OUT ? KP : 1];
    Piece<P::NO> po[VP];
    Piece<P::WITH == 2 ? 1 : 3> pw[P::DOT ? VP : 1];
    float pg = 1.f, pb = 0.f;
    const int nch = (int)((hi - lo + C - 1) / C);
    auto span = [&](int ch, int64_t& t0, int& n) {  // the chunk's first token and length, in processing order
        t0 = lo + (int64_t)(P::REV ? nch - 1 - ch : ch) * C;
        n = (int)(hi - t0 < C ? hi - t0 : C);
    };
    // Rows are read through buffers that begin at the chunk's first token and end behind its
    // last: a piece beyond it reads zeros, as does one beyond the row's width (offset FAR).
    // Backwards, row j is the chunk's token n - 1 - j; the offsets are those of a full
    // chunk, less the rows it lacks (negative ones wrap to beyond every buffer).
    auto row = [&](int j, int n) { return P::REV ? n - 1 - j : j; };
    auto rows = [&](const void* p, int64_t t0, int n, int width, uint32_t esz) {
        return make_rsrc(static_cast<const char*>(p) + (row0 + t0) * width * esz, (int64_t)n * width * esz);
    };
    uint32_t ek[KP], ev[VP], eo[NCT];  // elements into the buffers, or FAR
#pragma unroll
    for (int i = 0; i < KP; ++i) {
        const int e = tid + i * THR, j = e / (DKP / 8), q = e % (DKP / 8) * 8;
        ek[i] = j < C && q < a.DK ? (uint32_t)(row(j, C) * a.DK + q) : FAR;
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) {
        const int e = tid + i * THR, j = e / (SV / 8), q = e % (SV / 8) * 8;
        ev[i] = j < C && c0 + q < a.DV ? (uint32_t)(row(j, C) * a.DV + c0 + q) : FAR;
    }
#pragma unroll
    for (int c = 0; c < NCT; ++c) eo[c] = col[c] < a.DV ? (uint32_t)(row(4 * g4, C) * a.DV + col[c]) : FAR;
    const int step = P::REV ? -a.DV : a.DV;  // elements from one row of `out` to the next
    auto fetch = [&](int ch) {
        int64_t t0;
        int n;
        span(ch, t0, n);
        const rsrc_t rk = rows(a.kap, t0, n, a.DK, Piece<P::NK>::ESZ), ro = rows(a.omg, t0, n, a.DV, Piece<P::NO>::ESZ);
        const uint32_t lack = P::REV ? (uint32_t)(C - n) : 0u;
#pragma unroll
        for (int i = 0; i < KP; ++i) pk[i].load(rk, (ek[i] - lack * a.DK) * Piece<P::NK>::ESZ);
        if constexpr (P::OUT) {
            const rsrc_t rx = rows(a.xi, t0, n, a.DK, Piece<P::NX>::ESZ);
#pragma unroll
            for (int i = 0; i < KP; ++i) px[i].load(rx, (ek[i] - lack * a.DK) * Piece<P::NX>::ESZ);
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) po[i].load(ro, (ev[i] - lack * a.DV) * Piece<P::NO>::ESZ);
        if constexpr (P::DOT) {
            const rsrc_t rw = rows(a.with, t0, n, a.DV, P::WITH);
#pragma unroll
            for (int i = 0; i < VP; ++i) pw[i].load(rw, (ev[i] - lack * a.DV) * P::WITH);
        }
        pg = 1.f;
        pb = 0.f;
        const int j = w * 16 + m16;
        if (w < NT && j < n) {
            const int64_t t = t0 + row(j, n);
            if (!P::REV) pg = a.a[row0 + t];
            else if (t + 1 < a.T) pg = a.a[row0 + t + 1];
            if (!P::REV || P::OUT) pb = a.beta[row0 + t];
        }
    };
    float dg[4] = {0.f, 0.f, 0.f, 0.f};  // D_ts of diagonal block w: t = m16, s = 4 g4 + i
    // A chunk's decays, in set ch & 1: gates from the block's start through t, gates after s through its
    // end, b_s, o_t, the blocks' gates
    auto put = [&](int ch) {
        char* const buf = lds + (P::BUF == 2 && (ch & 1) ? P::ROWS : 0);
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int e = tid + i * THR, j = e / (DKP / 8), q = e % (DKP / 8) * 8;
            if (C * (DKP / 8) % THR != 0 && j >= C) continue;
            pk[i].store(buf + P::O_KA + j * P::RK + q * 2, P::PK);
            if constexpr (P::OUT) px[i].store(buf + P::O_XI + j * P::RK + q * 2, P::PK);
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            const int e = tid + i * THR, j = e / (SV / 8), q = e % (SV / 8) * 8;
            if (C * (SV / 8) % THR == 0 || j < C) {
                po[i].store(buf + P::O_OM + j * P::RV + q * 2, P::PV);
                if constexpr (P::DOT) pw[i].store_raw(buf + P::O_WI + j * P::RW + q * P::WITH);
            }
        }
        if (w < NT) {
            float* const d = dec + (ch & 1) * P::DEC;
            const float p = product_to(pg);  // every row of 16 lanes holds the block's gates
            const float q = product_from(__int_as_float(__builtin_amdgcn_update_dpp(0x3F800000, __float_as_int(pg), 0x101, 0xF, 0xF, false)));
            if constexpr (P::OUT) {
                // D_ts for s = 4 g4 + 3 is the product of the gates 4 g4 + 4 .. t; each smaller s takes one more
                float e = product_to(m16 >= 4 * g4 + 4 ? pg : 1.f);
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    dg[i] = m16 >= 4 * g4 + i ? e : 0.f;
                    const float g = __shfl(pg, 4 * g4 + i, 16);
                    e *= m16 >= 4 * g4 + i ? g : 1.f;
                }
            }
            int64_t t0;
            int n;
            span(ch, t0, n);
            if (lane < 16) {
                const int j = w * 16 + lane;
                d[j] = p;
                d[C + j] = q;
                d[2 * C + j] = P::REV ? (j < n ? 1.f : 0.f) : pb;
                d[3 * C + j] = P::REV ? pb : 1.f;
                if (lane == 15) d[4 * C + w] = p;
            }
        }
    };
    auto flush_dots = [&](int ch) {
        int64_t t0;
        int n;
        span(ch, t0, n);
        if (tid > C || (tid < C && tid >= n)) return;  // thread C: the sum of what the chunk's start gave
        const float* const f = dots + (ch & 1) * NW * (C + 1) + tid;
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) d += f[i * (C + 1)];
        const int64_t u = (int64_t)slab * a.NS + s;
        if (tid < C) a.dot[u * a.T + t0 + row(tid, n)] = d;
        else a.inter[u * a.nchunk + t0 / C] = d;
    };

    fetch(0);
    put(0);
    if (nch > 1) fetch(1);
    __syncthreads();
    float segdec = 1.f;
    for (int ch = 0; ch < nch; ++ch) {
        const char* const buf = lds + (P::BUF == 2 && (ch & 1) ? P::ROWS : 0);
        const char* const Ka = buf + P::O_KA;
        const char* const Om = buf + P::O_OM;
        const char* const Xi = buf + P::O_XI;
        const float* const fpre = dec + (ch & 1) * P::DEC;
        const float* const fsuf = fpre + C;
        const float* const fin = fsuf + C;
        const float* const fo = fin + C;
        const float tot0 = fo[C], tot1 = fo[C + 1], total = tot0 * tot1;
        // `with` at rows 16 t + 4 g4 + i of this lane's column (bf16: by a transposing read)
        auto with = [&](int t, int c, float (&v)[4]) {
            const char* const p = buf + P::O_WI + (t * 16 + 4 * g4) * P::RW + (w * NCT + c) * 16 * P::WITH;
            if constexpr (P::WITH == 2) {
                const uint2 u = read_tr(p + (m16 >> 2) * P::RW + (m16 & 3) * 8);
                v[0] = bf_lo(u.x); v[1] = bf_hi(u.x); v[2] = bf_lo(u.y); v[3] = bf_hi(u.y);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const float*>(p + i * P::RW + m16 * 4);
            }
        };
        f32x4_t acc[P::OUT ? NT : 1][NCT];
        if constexpr (P::OUT) {
            // P^T = kap xi^T, scaled: a tile (s block st, t block tt) a wavefront, its planes stored as
            // the operand of the product with omg (wavefront b takes diagonal tile b, whose decays it has)
            if (w < P::TILES) {
                const int tt = w == 0 ? 0 : 1, st = w == 1 ? 1 : 0;
                f32x4_t p = {0.f, 0.f, 0.f, 0.f};
                const char* const kr = Ka + (st * 16 + m16) * P::RK + g4 * 16;
                const char* const xr = Xi + (tt * 16 + m16) * P::RK + g4 * 16;
#pragma unroll
                for (int k2 = 0; k2 < DKP * 2; k2 += 64) {
                    uint4 ka[P::NK], xb[P::NX];
#pragma unroll
                    for (int i = 0; i < P::NK; ++i) ka[i] = *reinterpret_cast<const uint4*>(kr + i * P::PK + k2);
#pragma unroll
                    for (int i = 0; i < P::NX; ++i) xb[i] = *reinterpret_cast<const uint4*>(xr + i * P::PK + k2);
                    mma<P::NK, P::NX>(ka, xb, p);
                }
                const float4 in = *reinterpret_cast<const float4*>(fin + st * 16 + 4 * g4);
                float f[4] = {in.x, in.y, in.z, in.w};
                if (w < NT) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] *= dg[i];
                } else {
                    const float4 sf = *reinterpret_cast<const float4*>(fsuf + st * 16 + 4 * g4);
                    const float pr = fpre[tt * 16 + m16];
                    f[0] *= sf.x * pr; f[1] *= sf.y * pr; f[2] *= sf.z * pr; f[3] *= sf.w * pr;
                }
                uint2 o[3];
                split2(p[0] * f[0], p[1] * f[1], o[0].x, o[1].x, o[2].x);
                split2(p[2] * f[2], p[3] * f[3], o[0].y, o[1].y, o[2].y);
                char* const to = Pf + (tt + st) * 3 * 512 + lane * 8;  // tiles (0,0), (1,0), (1,1)
#pragma unroll
                for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(to + i * 512) = o[i];
            }
            if constexpr (P::DOT)
                if (ch > 0) flush_dots(ch - 1);
            // xi X_start
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < NCT; ++c) acc[t][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < DKT / 2; ++p) {
                uint4 xb[NCT][3];
#pragma unroll
                for (int c = 0; c < NCT; ++c) {
                    const float v[8] = {X[2 * p][c][0], X[2 * p][c][1], X[2 * p][c][2], X[2 * p][c][3],
                                        X[2 * p + 1][c][0], X[2 * p + 1][c][1], X[2 * p + 1][c][2], X[2 * p + 1][c][3]};
                    split8(v, xb[c]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    uint4 xa[P::NX];
#pragma unroll
                    for (int i = 0; i < P::NX; ++i)
                        xa[i] = *reinterpret_cast<const uint4*>(Xi + i * P::PK + (t * 16 + m16) * P::RK + p * 64 + g4 * 16);
#pragma unroll
                    for (int c = 0; c < NCT; ++c) mma<P::NX, 3>(xa, xb[c], acc[t][c]);
                }
            }
            float inter = 0.f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float4 pr = *reinterpret_cast<const float4*>(fpre + t * 16 + 4 * g4);
                const float q = t ? tot0 : 1.f;
                const float f[4] = {pr.x * q, pr.y * q, pr.z * q, pr.w * q};
#pragma unroll
                for (int c = 0; c < NCT; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][c][i] *= f[i];
                if constexpr (P::DOT) {  // what the chunk's start gives to xi_t X_t . with_t, summed over the chunk
                    const float4 o4 = *reinterpret_cast<const float4*>(fo + t * 16 + 4 * g4);
                    const float o[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
                    for (int c = 0; c < NCT; ++c) {
                        float v[4];
                        with(t, c, v);
#pragma unroll
                        for (int i = 0; i < 4; ++i) inter = fmaf(P::REV ? acc[t][c][i] * o[i] : acc[t][c][i], v[i], inter);
                    }
                }
            }
            if constexpr (P::DOT) {
                inter = wave_sum(inter);
                if (lane == 0) dots[((ch & 1) * NW + w) * (C + 1) + C] = inter;
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < DKT; ++k)
#pragma unroll
            for (int c = 0; c < NCT; ++c) X[k][c] *= total;
        // over the tokens
        uint4 om[NCT][P::NO], ow[NCT][3];
        float f[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 sf = *reinterpret_cast<const float4*>(fsuf + h * 16 + 4 * g4);
            const float4 in = *reinterpret_cast<const float4*>(fin + h * 16 + 4 * g4);
            const float q = h ? 1.f : tot1;
            f[4 * h] = sf.x * in.x * q; f[4 * h + 1] = sf.y * in.y * q;
            f[4 * h + 2] = sf.z * in.z * q; f[4 * h + 3] = sf.w * in.w * q;
        }
#pragma unroll
        for (int c = 0; c < NCT; ++c) {
#pragma unroll
            for (int i = 0; i < P::NO; ++i) {
                const char* o = Om + i * P::PV + (4 * g4 + (m16 >> 2)) * P::RV + ((w * NCT + c) * 16 + (m16 & 3) * 4) * 2;
                const uint2 x = read_tr(o), y = read_tr(o + 16 * P::RV);
                om[c][i] = make_uint4(x.x, x.y, y.x, y.y);
            }
            const uint32_t u[4] = {om[c][0].x, om[c][0].y, om[c][0].z, om[c][0].w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf_lo(u[i]);
                v[2 * i + 1] = bf_hi(u[i]);
            }
            if constexpr (P::NO == 3) {  // the planes' sum is the value
                const uint32_t m[4] = {om[c][1].x, om[c][1].y, om[c][1].z, om[c][1].w};
                const uint32_t l[4] = {om[c][2].x, om[c][2].y, om[c][2].z, om[c][2].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] += bf_lo(m[i]) + bf_lo(l[i]);
                    v[2 * i + 1] += bf_hi(m[i]) + bf_hi(l[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= f[i];
            split8(v, ow[c]);
        }
        if constexpr (P::OUT) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint4 pa[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const char* p = Pf + (t * 3 + i) * 512 + lane * 8;
                    const uint2 x = *reinterpret_cast<const uint2*>(p);
                    const uint2 y = t ? *reinterpret_cast<const uint2*>(p + 3 * 512) : make_uint2(0u, 0u);
                    pa[i] = make_uint4(x.x, x.y, y.x, y.y);
                }
#pragma unroll
                for (int c = 0; c < NCT; ++c) mma<3, P::NO>(pa, om[c], acc[t][c]);
            }
        }
#pragma unroll
        for (int k = 0; k < DKT; ++k) {
            uint4 ka[P::NK];
#pragma unroll
            for (int i = 0; i < P::NK; ++i) {
                const char* o = Ka + i * P::PK + (4 * g4 + (m16 >> 2)) * P::RK + (P::OUT ? 32 * (k >> 1) + 8 * (m16 & 3) + 4 * (k & 1) : 16 * k + 4 * (m16 & 3)) * 2;
                const uint2 x = read_tr(o), y = read_tr(o + 16 * P::RK);
                ka[i] = make_uint4(x.x, x.y, y.x, y.y);
            }
#pragma unroll
            for (int c = 0; c < NCT; ++c) mma<P::NK, 3>(ka, ow[c], X[k][c]);
        }
        if constexpr (P::OUT) {
            int64_t t0;
            int n;
            span(ch, t0, n);
            const rsrc_t rout = rows(a.out, t0, n, a.DV, 4);
            const int lack = P::REV ? (C - n) * a.DV : 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float4 o4 = *reinterpret_cast<const float4*>(fo + t * 16 + 4 * g4);
                const float o[4] = {o4.x, o4.y, o4.z, o4.w};
                float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < NCT; ++c) {
                    float v[4];
                    if constexpr (P::DOT) with(t, c, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        st_f1(P::REV ? acc[t][c][i] * o[i] : acc[t][c][i], rout, (eo[c] + (t * 16 + i) * step - lack) * 4u, 0);
                        if constexpr (P::DOT) d[i] = fmaf(acc[t][c][i], v[i], d[i]);
                    }
                }
                if constexpr (P::DOT)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[i] = ror_add<1>(ror_add<2>(ror_add<4>(ror_add<8>(d[i]))));
                        if (m16 == 0) dots[((ch & 1) * NW + w) * (C + 1) + t * 16 + 4 * g4 + i] = d[i];
                    }
            }
        } else {
            segdec *= total;
        }
        if (ch + 1 < nch) {
            if (P::BUF == 1) __syncthreads();
            put(ch + 1);
            if (ch + 2 < nch) fetch(ch + 2);
        }
        __syncthreads();
    }
    if constexpr (P::DOT) flush_dots(nch - 1);
    if (a.Xend) {
#pragma unroll
        for (int k = 0; k < DKT; ++k)
#pragma unroll
            for (int c = 0; c < NCT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = (P::OUT ? 32 * (k >> 1) + 8 * g4 + 4 * (k & 1) : 16 * k + 4 * g4) + i;
                    if (r < a.DK && col[c] < a.DV) a.Xend[state + r * (int64_t)a.DV + col[c]] = X[k][c][i];
                }
    }
    if (!P::OUT && slab == 0 && tid == 0) a.segdec[seg * a.NS + s] = segdec;
}

// Workgroups of the same stream and segment go to one XCD, one after the other
// (their rows are largely the same).
template <class P>
__global__ __launch_bounds__(P::THR, 2) void dense_pass_kernel(DenseArgs a) {
    extern __shared__ __align__(16) char lds[];
    int64_t us;
    int slab;
    block_unit((int)blockIdx.x, a.NS * a.nseg, a.nslab, us, slab);
    if (us < a.NS * a.nseg) dense_pass<P>(a, us, slab, lds);
}

constexpr int max2(int a, int b) { return a > b ? a : b; }

// Two or three passes in one launch: a's slabs, then b's, then c's.
template <class P1, class P2>
__global__ __launch_bounds__(P1::THR, 2) void dense_two_kernel(DenseArgs a, DenseArgs b) {
    static_assert(P1::THR == P2::THR, "one launch");
    extern __shared__ __align__(16) char lds[];
    int64_t us;
    int u;
    block_unit((int)blockIdx.x, a.NS * a.nseg, a.nslab + b.nslab, us, u);
    if (us >= a.NS * a.nseg) return;
    if (u < a.nslab) dense_pass<P1>(a, us, u, lds);
    else dense_pass<P2>(b, us, u - a.nslab, lds);
}
template <class P1, class P2, class P3>
__global__ __launch_bounds__(P1::THR, 2) void dense_three_kernel(DenseArgs a, DenseArgs b, DenseArgs c) {
    static_assert(P1::THR == P2::THR && P1::THR == P3::THR, "one launch");
    extern __shared__ __align__(16) char lds[];
    int64_t us;
    int u;
    block_unit((int)blockIdx.x, a.NS * a.nseg, a.nslab + b.nslab + c.nslab, us, u);
    if (us >= a.NS * a.nseg) return;
    if (u < a.nslab) dense_pass<P1>(a, us, u, lds);
    else if (u < a.nslab + b.nslab) dense_pass<P2>(b, us, u - a.nslab, lds);
    else dense_pass<P3>(c, us, u - a.nslab - b.nslab, lds);
}

template <class P>
DenseArgs dense_slabs(DenseArgs a) {
    a.nslab = (a.DV + P::SV - 1) / P::SV;
    a.nchunk = (a.T + P::C - 1) / P::C;
    return a;
}
template <class P>
hipError_t launch_passes(const DenseArgs& a0, hipStream_t st) {
    const DenseArgs a = dense_slabs<P>(a0);
    hipLaunchKernelGGL(dense_pass_kernel<P>, dim3((unsigned)unit_grid(a.NS * a.nseg, a.nslab)), dim3(P::THR), P::LDS, st, a);
    return hipGetLastError();
}
template <class P1, class P2>
hipError_t launch_passes(const DenseArgs& a0, const DenseArgs& b0, hipStream_t st) {
    const DenseArgs a = dense_slabs<P1>(a0), b = dense_slabs<P2>(b0);
    hipLaunchKernelGGL((dense_two_kernel<P1, P2>), dim3((unsigned)unit_grid(a.NS * a.nseg, a.nslab + b.nslab)), dim3(P1::THR),
                       max2(P1::LDS, P2::LDS), st, a, b);
    return hipGetLastError();
}
template <class P1, class P2, class P3>
hipError_t launch_passes(const DenseArgs& a0, const DenseArgs& b0, const DenseArgs& c0, hipStream_t st) {
    const DenseArgs a = dense_slabs<P1>(a0), b = dense_slabs<P2>(b0), c = dense_slabs<P3>(c0);
    hipLaunchKernelGGL((dense_three_kernel<P1, P2, P3>), dim3((unsigned)unit_grid(a.NS * a.nseg, a.nslab + b.nslab + c.nslab)),
                       dim3(P1::THR), max2(P1::LDS, max2(P2::LDS, P3::LDS)), st, a, b, c);
    return hipGetLastError();
}

// Columns a workgroup: 64, or 128 where there are that many (the products over
// the contracted width are then done once for all of them).
constexpr int dense_slab(int dv) { return dv <= 64 ? 64 : 128; }

// f(contracted width's tiles, column tiles a wavefront, wavefronts), for a pass of its own.
// Four wavefronts of 32 columns read each operand half as often as eight of 16, and hold
// twice the state (128 x 128, bf16: 4x8x8192 tokens 147 / 157 us, 1x8x131072 506 / 533; with fp32
// rows 291 / 282, 1x8x32768 302 / 294); from 128 to 256 rows of state a lane's registers allow 16 columns.
template <int N>
using Int = std::integral_constant<int, N>;
template <class F>
hipError_t dense_sized(int DK, int DV, F f) {
    const bool wide = dense_slab(DV) == 128;
    if (DK <= 64) return wide ? f(Int<4>{}, Int<2>{}, Int<4>{}) : f(Int<4>{}, Int<1>{}, Int<4>{});
    if (DK <= 128) return wide ? f(Int<8>{}, Int<2>{}, Int<4>{}) : f(Int<8>{}, Int<1>{}, Int<4>{});
    return wide ? f(Int<16>{}, Int<1>{}, Int<8>{}) : f(Int<16>{}, Int<1>{}, Int<4>{});
}

template <int NX, int NK, int NO>
hipError_t dense_y(const DenseArgs& a, hipStream_t st) {
    return dense_sized(a.DK, a.DV, [&](auto t, auto c, auto w) {
        return launch_passes<DensePass<t(), c(), w(), NX, NK, NO, true, false, false>>(a, st);
    });
}
template <int NK, int NO>
hipError_t dense_s(const DenseArgs& a, hipStream_t st) {
    return dense_sized(a.DK, a.DV, [&](auto t, auto c, auto w) {
        return launch_passes<DensePass<t(), c(), w(), 1, NK, NO, false, false, false>>(a, st);
    });
}
// the segments' own S and G (kap planes NK, and omg planes of S and of G)
template <int NK, int NOS, int NOG>
hipError_t dense_sg(const DenseArgs& s, const DenseArgs& g, hipStream_t st) {
    return dense_sized(s.DK, s.DV, [&](auto t, auto c, auto w) {
        return launch_passes<DensePass<t(), c(), w(), 1, NK, NOS, false, false, false>,
                             DensePass<t(), c(), w(), 1, NK, NOG, false, true, false>>(s, g, st);
    });
}
// dq, dk and dv: NR planes of the rows q, k and v, three of dy's. dq and dk contract the
// value width (tiles TV) and put out the key width; dv the other way round (tiles TK). In one
// launch all have 4 wavefronts, or 8 where a width passes 128, or where fp32 rows of 128 leave
// room for one workgroup on a CU (2x8x4096 tokens, fp32, all of the backward, with 4 / 8: 128 x 128
// 304 / 261 us, 64 x 128 201 / 217, 64 x 64 100 / 144).
template <int NR, int TK, int TV>
hipError_t dense_grads_t(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st) {
    constexpr int W = TK == 16 || TV == 16 || (NR == 3 && TK == 8 && TV == 8) ? 8 : 4;
    constexpr int CK = W == 8 || TK == 4 ? 1 : 2, CV = W == 8 || TV == 4 ? 1 : 2;  // column tiles a wavefront
    return launch_passes<DensePass<TV, CK, W, 3, NR, NR, true, false, true>, DensePass<TV, CK, W, NR, 3, NR, true, true, true>,
                         DensePass<TK, CV, W, NR, NR, 3, true, true, false>>(q, k, v, st);
}
template <int NR>
hipError_t dense_grads(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st) {
    auto tiles = [](int d, auto f) { return d <= 64 ? f(Int<4>{}) : d <= 128 ? f(Int<8>{}) : f(Int<16>{}); };
    return tiles(v.DK, [&](auto tk) {
        return tiles(q.DK, [&](auto tv) { return dense_grads_t<NR, tk(), tv()>(q, k, v, st); });
    });
}

}  // namespace
}  // namespace sdm
