// conv.hip -- the short causal convolution over time of every channel, and its gradients, on gfx950:
//   z_t = bias + sum_j w_j x_{t-K+1+j},   y_t = z_t or silu(z_t) = z_t sigmoid(z_t),
// over [B, H, T, d] tokens (heads of any stride), K from 2 to 8 taps, the K - 1 inputs before token 0
// from a state and those behind the last token into it. Backward, with dz_t = dy_t silu'(z_t):
//   dx_t = sum_j w_j dz_{t+K-1-j},   dw_j = sum_t dz_t x_{t-K+1+j},   dbias = sum_t dz_t.
//
// A thread owns VEC channels (a piece of a row, or one channel where rows are not aligned to pieces) over a
// tile of tokens, a wavefront 64 such threads of one tile, so that lengths and begins of sequences are scalar:
// the last K - 1 inputs and the weights stay in registers, and each input is read once from HBM (a tile's first K - 1
// inputs also by the tile before, out of the L2). HBM-bound: 4 x 8192 x 2048 in bf16 with 4 taps, forward 54 to 58 us in the
// kernel and 61 a call over inputs in turn (269 MB, 4.4 TB/s; a copy of that card 5.15), backward 98 (403 MB); pieces of 8
// elements forwards (16 bytes), 4 backwards, where each channel holds 3 K + 2 floats; narrower where sizes, strides or
// addresses need it (4 x 8192, forward: 2044 channels in pieces of 4 61 us, 77 one by one; 2047 one by one
// 81, 90 in rows of odd strides; in fp32 2048 channels 108, backward 169).
// One token of 256 sequences: 6.3 us, and 8.9 a call (the host's side).
#include <type_traits>

#include "sdm_internal.h"
#include "sdm_rows.h"

namespace sdm {
namespace {

constexpr int AHEAD = 4;  // tokens whose loads are in flight together

// The tile that a wavefront works on, and the thread's channels in it
struct ConvAt {
    int c, h;
    int64_t b, t0, t1;
    bool ok;
};
template <int VEC, typename Args>
__device__ __forceinline__ ConvAt conv_at(const Args& a) {
    ConvAt w;
    uint32_t i = blockIdx.x;  // [b][tile][64 threads of the pieces of all heads]
    const uint32_t v = i % (uint32_t)a.groups * 64u + threadIdx.x;
    i /= (uint32_t)a.groups;
    w.ok = v < (uint32_t)(a.H * a.nvec);
    w.c = (int)(v % (uint32_t)a.nvec) * VEC;
    w.h = (int)(v / (uint32_t)a.nvec);
    w.t0 = (int64_t)(i % (uint32_t)a.ntile) * a.tile;
    w.b = i / (uint32_t)a.ntile;
    w.t1 = w.t0 + a.tile < a.T ? w.t0 + a.tile : a.T;
    return w;
}

__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t T) {
    if (!lengths) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n > T ? T : n;
}

// Sums over up to 7 rounded products in the taps' order; silu by the hardware's exponential and reciprocal
template <int K, int VEC>
__device__ __forceinline__ void taps(const float (&w)[K][VEC], const float (&bias)[VEC], const float (&x)[K][VEC], float (&z)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        z[i] = bias[i];
#pragma unroll
        for (int j = 0; j < K; ++j) z[i] = fmaf(w[j][i], x[j][i], z[i]);
    }
}

template <int VEC>
__device__ __forceinline__ void clear(float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = 0.f;
}

// The piece's VEC * K weights lie one after another
template <int K, int VEC, typename Args>
__device__ __forceinline__ void load_weights(const Args& a, int h, int c, float (&w)[K][VEC], float (&bias)[VEC]) {
    const int64_t row = (int64_t)h * a.d + c;
    float all[VEC * K];
    load_piece<VEC * K, false>(a.w, row * K, all);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][i] = all[i * K + j];
    clear<VEC>(bias);
    if (a.bias) load_piece<VEC, false>(a.bias, row, bias);
}

// The state's row m (token m - (K - 1)); zeros without a state
template <int K, int VEC, bool BF16>
__device__ __forceinline__ void load_state(const void* S0, int64_t bh, int d, int c, int m, float (&v)[VEC]) {
    if (S0) {
        load_piece<VEC, BF16>(S0, (bh * (K - 1) + m) * d + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = 0.f;
    }
}

// The window win[0 .. K - 1]: the newest input last
template <int K, int VEC>
__device__ __forceinline__ void push(float (&win)[K][VEC], const float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) win[K - 1][i] = x[i];
}
template <int K, int VEC>
__device__ __forceinline__ void pop(float (&win)[K][VEC]) {
#pragma unroll
    for (int m = 0; m < K - 1; ++m)
#pragma unroll
        for (int i = 0; i < VEC; ++i) win[m][i] = win[m + 1][i];
}

// The K - 1 inputs in front of token t0, as token t0 sees them: none of a sequence that ended
template <int K, int VEC, bool BF16, typename Args>
__device__ __forceinline__ void window(const Args& a, const ConvAt& w, int64_t n, const void* x, float (&win)[K][VEC]) {
#pragma unroll
    for (int m = 0; m < K - 1; ++m) {
        const int64_t t = w.t0 - (K - 1) + m;
        if (t < 0) load_state<K, VEC, BF16>(a.S0, w.b * a.H + w.h, a.d, w.c, (int)(t + K - 1), win[m]);
        else if (t < n) load_piece<VEC, BF16>(x, t * a.x_t, win[m]);
        else clear<VEC>(win[m]);
        if (a.start && t >= 0 && t < n && a.start[w.b * a.T + t])
#pragma unroll
            for (int k = 0; k < m; ++k) clear<VEC>(win[k]);
    }
}

template <int K, int VEC, bool BF16>
__global__ __launch_bounds__(64) void conv_kernel(ConvArgs a) {
    const ConvAt at = conv_at<VEC>(a);
    if (!at.ok) return;
    const int64_t n = length_of(a.lengths, at.b, a.T), bh = at.b * a.H + at.h;
    const char* x = static_cast<const char*>(a.x) + (at.b * a.x_b + at.h * a.x_h + at.c) * (BF16 ? 2 : 4);
    const uint8_t* start = a.start ? a.start + at.b * a.T : nullptr;
    float w[K][VEC], bias[VEC], win[K][VEC];
    load_weights<K, VEC>(a, at.h, at.c, w, bias);
    window<K, VEC, BF16>(a, at, n, x, win);
    // The state behind the last token, by the thread that holds the state in front of the first one (which it
    // may overwrite): rows of tokens n - (K - 1) .. n - 1, zeros in front of the last sequence's first token
    if (a.S && at.t0 == 0) {
        float S0[K][VEC];
        int64_t first = -K;
#pragma unroll
        for (int m = 0; m < K - 1; ++m) {
            load_state<K, VEC, BF16>(a.S0, bh, a.d, at.c, m, S0[m]);
            const int64_t t = n - (K - 1) + m;
            if (start && t >= 0 && start[t]) first = t;
        }
#pragma unroll
        for (int m = 0; m < K - 1; ++m) {
            const int64_t t = n - (K - 1) + m;
            float v[VEC];
            clear<VEC>(v);
            if (t >= first) {
                if (t >= 0) {
                    load_piece<VEC, BF16>(x, t * a.x_t, v);
                } else {
#pragma unroll
                    for (int k = 0; k < K - 1; ++k)
                        if (t + K - 1 == k)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) v[i] = S0[k][i];
                }
            }
            store_piece<VEC, BF16>(a.S, (bh * (K - 1) + m) * a.d + at.c, v);
        }
    }
    const int64_t out = bh * a.T * a.d + at.c, e = at.t1 < n ? at.t1 : n;
    int64_t t = at.t0;
    for (; t < e; t += AHEAD) {  // the loads of AHEAD tokens before the first one's sums (stores may not pass them)
        float xs[AHEAD][VEC];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) load_piece<VEC, BF16>(x, (t + k < e ? t + k : e - 1) * a.x_t, xs[k]);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (t + k >= e) break;
            if (start && start[t + k])
#pragma unroll
                for (int m = 0; m < K - 1; ++m) clear<VEC>(win[m]);
            push<K, VEC>(win, xs[k]);
            float z[VEC];
            taps<K, VEC>(w, bias, win, z);
            if (a.silu)
#pragma unroll
                for (int i = 0; i < VEC; ++i) z[i] *= sigmoid(z[i]);
            store_piece<VEC, BF16>(a.y, out + (t + k) * a.d, z);
            pop<K, VEC>(win);
        }
    }
    if (t > e) t = e > at.t0 ? e : at.t0;
    float none[VEC];
    clear<VEC>(none);
    for (; t < at.t1; ++t) store_piece<VEC, BF16>(a.y, out + t * a.d, none);
}

// A tile walks its tokens and the K - 1 behind them; dx of a token is complete K - 1 tokens later.
// Its share of dw and dbias goes to a row of `part` [B * ntile][K + 1][H * d].
template <int K, int VEC, bool BF16>
__global__ __launch_bounds__(64, 2) void conv_bwd_kernel(ConvBwdArgs a) {
    const ConvAt at = conv_at<VEC>(a);
    if (!at.ok) return;
    const int64_t n = length_of(a.lengths, at.b, a.T), bh = at.b * a.H + at.h;
    const char* x = static_cast<const char*>(a.x) + (at.b * a.x_b + at.h * a.x_h + at.c) * (BF16 ? 2 : 4);
    const uint8_t* start = a.start ? a.start + at.b * a.T : nullptr;
    const int64_t dxo = at.b * a.dx_b + at.h * a.dx_h + at.c;
    float w[K][VEC], bias[VEC], win[K][VEC], dw[K][VEC], db[VEC], dx[K][VEC];
    load_weights<K, VEC>(a, at.h, at.c, w, bias);
    window<K, VEC, BF16>(a, at, n, x, win);
    clear<VEC>(db);
#pragma unroll
    for (int j = 0; j < K; ++j) {
        clear<VEC>(dw[j]);
        clear<VEC>(dx[j]);
    }
    int64_t first = -K;  // the last sequence's first token among those seen
    // (a start in the tile's last K - 1 tokens before t0 cannot part token t0 from the state: no need to look)
    const int64_t end = at.t1 + K - 1;
    // AHEAD tokens from t8 on; with ALL, all of them are there (loads without a branch stay in flight together)
    struct Group {
        Piece<VEC, BF16> x[AHEAD], dy[AHEAD];
    };
    auto fetch = [&](auto whole, int64_t t8) {
        constexpr bool ALL = decltype(whole)::value;
        Group f{};
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (ALL || (t8 + k < n && t8 + k < end)) {
                f.x[k].load(x, (t8 + k) * a.x_t);
                f.dy[k].load(a.dy, (bh * a.T + t8 + k) * a.d + at.c);
            }
        return f;
    };
    auto group = [&](auto whole, const Group& f, int64_t t8) {
        constexpr bool ALL = decltype(whole)::value;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int64_t t = t8 + k;
            if (!ALL && t >= end) break;
            float dz[VEC], xs[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                dz[i] = f.dy[k][i];
                xs[i] = f.x[k][i];
            }
            if (ALL || t < n) {
                if (start && start[t]) {
                    first = t;
#pragma unroll
                    for (int m = 0; m < K - 1; ++m) clear<VEC>(win[m]);
                }
                push<K, VEC>(win, xs);
                if (a.silu) {
                    float z[VEC];
                    taps<K, VEC>(w, bias, win, z);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float s = sigmoid(z[i]);
                        dz[i] *= s * fmaf(z[i], 1.f - s, 1.f);
                    }
                }
                if (t < at.t1)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        db[i] += dz[i];
#pragma unroll
                        for (int j = 0; j < K; ++j) dw[j][i] = fmaf(dz[i], win[j][i], dw[j][i]);
                    }
            }
            // dx[j] is that of token t - (K - 1) + j: it passed through tap j of token t, if in its sequence
            if (t - (K - 1) >= first) {
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) dx[j][i] = fmaf(w[j][i], dz[i], dx[j][i]);
            } else {
#pragma unroll
                for (int j = 0; j < K; ++j)
                    if (t - (K - 1) + j >= first)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) dx[j][i] = fmaf(w[j][i], dz[i], dx[j][i]);
            }
            const int64_t u = t - (K - 1);  // complete
            if (u >= at.t0 || u < 0) {
                if (a.dS && u < n && u > n - K && u >= first) {  // it is in the last state too
                    float g[VEC];
                    load_piece<VEC, BF16>(a.dS, (bh * (K - 1) + u - n + K - 1) * a.d + at.c, g);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) dx[0][i] += g[i];
                }
                if (u >= 0) store_piece<VEC, BF16>(a.dx, dxo + u * a.dx_t, dx[0]);
                else if (a.dS0) store_piece<VEC, BF16>(a.dS0, (bh * (K - 1) + t) * a.d + at.c, dx[0]);
            }
            pop<K, VEC>(win);
            pop<K, VEC>(dx);
            clear<VEC>(dx[K - 1]);
        }
    };
    int64_t t = at.t0;
    const int64_t e = end < n ? end : n;
    if (BF16 && t + AHEAD <= e) {  // a group ahead (130 -> 98 us at 4 x 8192 x 2048; in fp32 it takes 61 registers and a wavefront's room a SIMD)
        Group f = fetch(std::true_type{}, t);
        for (; t + 2 * AHEAD <= e; t += AHEAD) {
            const Group next = fetch(std::true_type{}, t + AHEAD);
            group(std::true_type{}, f, t);
            f = next;
        }
        group(std::true_type{}, f, t);
        t += AHEAD;
    }
    for (; t + AHEAD <= e; t += AHEAD) group(std::true_type{}, fetch(std::true_type{}, t), t);
    for (; t < end; t += AHEAD) group(std::false_type{}, fetch(std::false_type{}, t), t);
    const int64_t hd = (int64_t)a.H * a.d, row = (at.b * a.ntile + at.t0 / a.tile) * (K + 1) * hd + (int64_t)at.h * a.d + at.c;
#pragma unroll
    for (int j = 0; j < K; ++j) store_piece<VEC, false>(a.part, row + j * hd, dw[j]);
    store_piece<VEC, false>(a.part, row + K * hd, db);
}

// dw [H * d][K] and dbias [H * d] of the columns' sums
struct ConvSums {
    float* dw; float* db;
    int K;
    int64_t hd;
    __device__ void operator()(int64_t i, float v) const {
        const int64_t j = i / hd, c = i - j * hd;
        if (j < K) dw[c * K + j] = v;
        else if (db) db[c] = v;
    }
};

// Tokens a tile: so many that the wavefronts (of 64 pieces of `vec` channels) fill the SIMDs once, within bounds.
// Forwards 4 wavefronts fit a SIMD and short tiles cost little (4 x 8192 x 2048: 54 us by tiles of 16 or 32, 55 by 128);
// backwards 2, a tile reads K - 1 tokens more and leaves a row of sums, and a second round of few wavefronts would cost as
// much as a full one (125 us by tiles of 64, 98 by the 64 x 2048 that fill the SIMDs once).
// At least 8 tokens, so that only the first tile reads the state.
int64_t tile_of(int64_t B, int64_t H, int64_t T, int64_t d, int vec, int slots, int most) {
    const int64_t waves = B * ((H * d + 64 * vec - 1) / (64 * vec)), want = waves < slots ? slots / waves : 1;
    int64_t t = (T + want - 1) / want;
    t = (t + AHEAD - 1) / AHEAD * AHEAD;
    return t < CONV_TILE_MIN ? CONV_TILE_MIN : t > most ? most : t;
}
static_assert(CONV_TILE_MIN >= 7, "");

template <int K, int VEC, bool BF16>
void conv_go(const ConvArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((conv_kernel<K, VEC, BF16>), dim3((unsigned)(a.B * a.ntile * a.groups)), dim3(64), 0, st, a);
}
template <int K, int VEC, bool BF16>
void conv_go(const ConvBwdArgs& a, hipStream_t st) {
    hipLaunchKernelGGL((conv_bwd_kernel<K, VEC, BF16>), dim3((unsigned)(a.B * a.ntile * a.groups)), dim3(64), 0, st, a);
}
template <int VEC, bool BF16, typename A>
void conv_taps(A& a, hipStream_t st) {
    a.nvec = a.d / VEC;
    a.groups = (int)((a.H * a.nvec + 63) / 64);
    switch (a.K) {
        case 2: conv_go<2, VEC, BF16>(a, st); break;
        case 3: conv_go<3, VEC, BF16>(a, st); break;
        case 4: conv_go<4, VEC, BF16>(a, st); break;
        case 5: conv_go<5, VEC, BF16>(a, st); break;
        case 6: conv_go<6, VEC, BF16>(a, st); break;
        case 7: conv_go<7, VEC, BF16>(a, st); break;
        default: conv_go<8, VEC, BF16>(a, st);
    }
}

int64_t tiles(int64_t T, int64_t tile) { return T > tile ? (T + tile - 1) / tile : 1; }

int64_t bwd_tile(int64_t B, int64_t H, int64_t T, int64_t d) { return tile_of(B, H, T, d, 4, 2048, 1024); }

}  // namespace

int64_t conv_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t d, int K) {
    return B * tiles(T, bwd_tile(B, H, T, d)) * (K + 1) * H * d * 4;
}

hipError_t launch_conv(ConvArgs a, hipStream_t st) {
    a.tile = (int)tile_of(a.B, a.H, a.T, a.d, 8, 4096, 32);
    a.ntile = tiles(a.T, a.tile);
    if (a.bf16) a.align >= 8 ? conv_taps<8, true>(a, st) : a.align >= 4 ? conv_taps<4, true>(a, st) : conv_taps<1, true>(a, st);
    else a.align >= 4 ? conv_taps<4, false>(a, st) : conv_taps<1, false>(a, st);
    return hipGetLastError();
}

hipError_t launch_conv_backward(ConvBwdArgs a, hipStream_t st) {
    a.tile = (int)bwd_tile(a.B, a.H, a.T, a.d);
    a.ntile = tiles(a.T, a.tile);
    if (a.bf16) a.align >= 4 ? conv_taps<4, true>(a, st) : conv_taps<1, true>(a, st);
    else a.align >= 4 ? conv_taps<4, false>(a, st) : conv_taps<1, false>(a, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t hd = (int64_t)a.H * a.d;
    return sum_columns(a.part, a.B * a.ntile, (a.K + 1) * hd, ConvSums{a.dw, a.dbias, a.K, hd}, st);
}

}  // namespace sdm
