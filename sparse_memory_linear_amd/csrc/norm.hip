// norm.hip -- RMS-Norm of a token's row with the residual's addition, and its
// gradients, on gfx950:
//   h = x + res,   y = h / sqrt(mean(h^2) + eps) * gamma,
// y in fp32, bf16 or e4m3 with fp32 scales (per row, or per group of columns).
// Backward, with r = 1 / sqrt(mean(h^2) + eps) and n = h r:
//   dx = dh + r (gamma dy - n mean(gamma dy n)),   dgamma = sum over rows of dy n.
//
// Both read each input once and write each output once: a row stays in the
// registers of the TPR threads that own it (NV pieces of VEC elements each),
// between its sums and its outputs. HBM-bound: 32768 rows of 1024 in bf16 with a
// residual, to bf16 and e4m3 with a scale per 128 columns, 236 MB in 50 us (4.7 TB/s; a
// copy of 1 GB reaches 4.75); the backward, 268 MB, in 58 us (4.6 TB/s). One row a thread
// group and no loop over rows: with 4 rows in turn the forward took 57 us in rotation, against 48.
//
// The norm is taken of the fp32 sum x + res; h is stored rounded to its type,
// and the backward works from the stored h, so that it reads no statistics.
#include "sdm_buffer.h"
#include "sdm_internal.h"

namespace sdm {
namespace {

constexpr int VEC = 8;

// A thread's piece: VEC consecutive elements of a row, n of which lie in it. Rows
// need not begin at a multiple of the piece's bytes (d odd): the vector types
// carry the elements' alignment only, which global memory accesses allow.
typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4a __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2b __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ void load_vec(const void* p, bool bf16, int64_t e, int n, float (&v)[VEC]) {
    if (bf16) {
        const uint16_t* b = static_cast<const uint16_t*>(p) + e;
        if (n >= VEC) {
            const u32x4a x = *reinterpret_cast<const u32x4a*>(b);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i < n ? __uint_as_float((uint32_t)b[i] << 16) : 0.f;
        }
    } else {
        const float* f = static_cast<const float*>(p) + e;
        if (n >= VEC) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const f32x4a x = *reinterpret_cast<const f32x4a*>(f + i);
                v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = i < n ? f[i] : 0.f;
        }
    }
}

// elements of the row from column c on (TAIL false: d a multiple of VEC, no partial pieces)
template <bool TAIL>
__device__ __forceinline__ int left(int d, int c) {
    return TAIL ? d - c : VEC;
}

// nearest even; a NaN stays one
__device__ __forceinline__ uint32_t to_bf16(float f) {
    const uint32_t u = __float_as_uint(f);
    if (f != f) return (u >> 16) | 0x40u;
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

__device__ __forceinline__ void store_vec(void* p, bool bf16, int64_t e, int n, const float (&v)[VEC]) {
    if (bf16) {
        uint16_t* b = static_cast<uint16_t*>(p) + e;
        if (n >= VEC) {
            uint32_t u[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC; i += 2) u[i / 2] = to_bf16(v[i]) | to_bf16(v[i + 1]) << 16;
            *reinterpret_cast<u32x4a*>(b) = u32x4a{u[0], u[1], u[2], u[3]};
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < n) b[i] = (uint16_t)to_bf16(v[i]);
        }
    } else {
        float* f = static_cast<float*>(p) + e;
        if (n >= VEC) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) *reinterpret_cast<f32x4a*>(f + i) = f32x4a{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (i < n) f[i] = v[i];
        }
    }
}

// v / scale in e4m3 (nearest even) with |v| <= 448 scale; 0 for a scale of 0. The codes are those of
// the fp32 quotient: a product with the scale's reciprocal is off by up to two steps, and a value in
// some 10^6, near the border of two codes, then falls to the other side. Each correction by the exact rest of
// the division leaves the nearest value to a quotient at most a step off (Markstein's theorem, for a
// reciprocal rounded to nearest); the first takes the product that near. (32768 x 1024, groups of 128:
// 44 us by the reciprocal alone, 45 so, 47 by divisions; 8192 x 8192, a scale a row: 89, 94, 100.)
// Tiny scales are raised first, with their values, so that the rests stay normal numbers.
__device__ __forceinline__ void store_e4m3(void* p, int64_t e, int n, const float (&v)[VEC], float scale) {
    uint8_t* b = static_cast<uint8_t*>(p) + e;
    const float up = scale < 0x1p-80f ? 0x1p60f : 1.f, s = scale * up, inv = scale == 0.f ? 0.f : 1.f / s;
    auto quotient = [&](float x) {
        x *= up;
        float q = x * inv;
        q = fmaf(fmaf(-q, s, x), inv, q);
        return fmaf(fmaf(-q, s, x), inv, q);
    };
    uint32_t u[VEC / 4];
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
        const int q = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i]), quotient(v[4 * i + 1]), 0, false);
        u[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[4 * i + 2]), quotient(v[4 * i + 3]), q, true);
    }
    if (n >= VEC) {
        *reinterpret_cast<u32x2b*>(b) = u32x2b{u[0], u[1]};
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (i < n) b[i] = (uint8_t)(u[i / 4] >> (8 * (i % 4)));
    }
}

// The scale that maps the largest magnitude onto e4m3's largest value, 448 (a product with
// 1 / 448 is a step off the quotient for more than half of all magnitudes). It
// stays a normal number; 0 for a row of zeros, NaN or infinite where the largest is.
__device__ __forceinline__ float e4m3_scale(float amax) {
    const float s = amax / 448.f;
    return amax == 0.f ? 0.f : s < 1.17549435e-38f ? 1.17549435e-38f : s;
}

// the larger of m >= 0 and |x|; a NaN of either stays (fmaxf drops it, and a row of NaN then has a scale of 0)
__device__ __forceinline__ float larger(float m, float x) { return __builtin_elementwise_maximum(m, fabsf(x)); }

// Sum and maximum over the TPR threads that own a row (the same on all of them)
template <int TPR>
__device__ __forceinline__ void row_reduce(float& sum, float& mx, float (*buf)[2]) {
    for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) {
        sum += __shfl_xor(sum, m);
        mx = larger(mx, __shfl_xor(mx, m));
    }
    if constexpr (TPR > 64) {
        const int w = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) { buf[w][0] = sum; buf[w][1] = mx; }
        __syncthreads();
        sum = 0.f; mx = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) { sum += buf[i][0]; mx = larger(mx, buf[i][1]); }
    }
}

template <int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    __shared__ float buf[TPR < 64 ? 1 : TPR / 64][2];
    const int lane = threadIdx.x % TPR;
    float ga[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * VEC;
        if (c < a.d) load_vec(a.gamma, false, c, left<TAIL>(a.d, c), ga[j]);
    }
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + threadIdx.x / TPR;
    if (row >= a.rows) return;  // TPR > 64: all of the workgroup's threads have this row
    float v[NV][VEC];
    const int64_t at = row * a.d;
    float ss = 0.f, mx = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * VEC;
        if (c >= a.d) break;
        load_vec(a.x, a.x_bf16, at + c, left<TAIL>(a.d, c), v[j]);
        if (a.res) {
            float r[VEC];
            load_vec(a.res, a.h_bf16, at + c, left<TAIL>(a.d, c), r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[j][i] += r[i];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * VEC;
        if (c >= a.d) break;
        if (a.res) store_vec(a.h, a.h_bf16, at + c, left<TAIL>(a.d, c), v[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            ss = fmaf(v[j][i], v[j][i], ss);
            v[j][i] *= ga[j][i];
            mx = larger(mx, v[j][i]);
        }
    }
    row_reduce<TPR>(ss, mx, buf);
    const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
    float scale = 0.f;
    if (a.y_type == NORM_E4M3 && a.group == 0) {
        scale = e4m3_scale(mx * r);
        if (lane == 0) a.scale[row] = scale;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * VEC;
        if constexpr (!TAIL) {  // (groups divide d, and are multiples of 8)
            if (a.y_type == NORM_E4M3 && a.group) {  // group / 8 neighbouring lanes share a scale
                float m = 0.f;
                if (c < a.d)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) m = larger(m, v[j][i] * r);
                for (int k = 1; k < a.group / 8; k <<= 1) m = larger(m, __shfl_xor(m, k));
                scale = e4m3_scale(m);
                if (c < a.d && c % a.group == 0) a.scale[row * (a.d / a.group) + c / a.group] = scale;
            }
        }
        if (c >= a.d) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] *= r;
        if (a.y_type == NORM_E4M3) store_e4m3(a.y, at + c, left<TAIL>(a.d, c), v[j], scale);
        else store_vec(a.y, a.y_type == NORM_BF16, at + c, left<TAIL>(a.d, c), v[j]);
    }
}

// A block's rows' share of dgamma stays in registers, its wavefronts' shares are
// added in order in LDS, and the blocks' rows of `part` by norm_dgamma_kernel:
// the order of all sums follows from the sizes alone.
template <int TPR, int NV, bool TAIL>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(NormBwdArgs a) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
    extern __shared__ float dg[];  // [d] (TPR < 256)
    __shared__ float buf[TPR < 64 ? 1 : TPR / 64][2];
    const int lane = threadIdx.x % TPR;
    float ga[NV][VEC], acc[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + lane) * VEC;
        if (c < a.d) load_vec(a.gamma, false, c, left<TAIL>(a.d, c), ga[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[j][i] = 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.rows; row += (int64_t)gridDim.x * RPB) {
        float h[NV][VEC], dy[NV][VEC];
        const int64_t at = row * a.d;
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + lane) * VEC;
            if (c >= a.d) break;
            load_vec(a.h, a.h_bf16, at + c, left<TAIL>(a.d, c), h[j]);
            load_vec(a.dy, a.g_bf16, at + c, left<TAIL>(a.d, c), dy[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + lane) * VEC;
            if (c >= a.d) break;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                ss = fmaf(h[j][i], h[j][i], ss);
                dot = fmaf(dy[j][i] * ga[j][i], h[j][i], dot);
            }
        }
        for (int m = 1; m < (TPR < 64 ? TPR : 64); m <<= 1) {
            ss += __shfl_xor(ss, m);
            dot += __shfl_xor(dot, m);
        }
        if constexpr (TPR > 64) {
            const int w = threadIdx.x >> 6;
            __syncthreads();
            if ((threadIdx.x & 63) == 0) { buf[w][0] = ss; buf[w][1] = dot; }
            __syncthreads();
            ss = 0.f; dot = 0.f;
#pragma unroll
            for (int i = 0; i < TPR / 64; ++i) { ss += buf[i][0]; dot += buf[i][1]; }
        }
        const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
        const float k = dot * r * r / (float)a.d;  // n mean(g dy n) = h (dot r^2 / d)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + lane) * VEC;
            if (c >= a.d) break;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                acc[j][i] = fmaf(dy[j][i], h[j][i] * r, acc[j][i]);
                o[i] = r * (dy[j][i] * ga[j][i] - h[j][i] * k);
            }
            if (a.dh) {
                float t[VEC];
                load_vec(a.dh, a.g_bf16, at + c, left<TAIL>(a.d, c), t);
#pragma unroll
                for (int i = 0; i < VEC; ++i) o[i] += t[i];
            }
            store_vec(a.dx, a.g_bf16, at + c, left<TAIL>(a.d, c), o);
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * a.d;
    if constexpr (TPR < 256) {
        for (int w = 0; w < RPB; ++w) {
            if (threadIdx.x / TPR == w)
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int c = (j * TPR + lane) * VEC;
                    if (c >= a.d) break;
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (c + i < a.d) dg[c + i] = w ? dg[c + i] + acc[j][i] : acc[j][i];
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += 256) part[c] = dg[c];
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * TPR + lane) * VEC;
            if (c >= a.d) break;
            store_vec(part, false, c, left<TAIL>(a.d, c), acc[j]);
        }
    }
}

// dgamma = the sum of the blocks' rows: 16 columns a workgroup, 64 groups of 16
// lanes each adding every 64th row, then the 64 sums pairwise.
__global__ __launch_bounds__(1024) void norm_dgamma_kernel(const float* part, float* dgamma, int blocks, int d) {
    __shared__ float s[64][17];
    const int l = threadIdx.x & 15, w = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
    float x = 0.f;
    if (c < d)
#pragma unroll 4
        for (int b = w; b < blocks; b += 64) x += part[(int64_t)b * d + c];
    s[w][l] = x;
    for (int n = 32; n > 0; n >>= 1) {
        __syncthreads();
        if (w < n) s[w][l] = x += s[w + n][l];
    }
    if (w == 0 && c < d) dgamma[c] = x;
}

template <int TPR, int NV, bool TAIL>
void norm_launch(const NormArgs& a, hipStream_t st) {
    constexpr int RPB = TPR < 256 ? 256 / TPR : 1, THR = TPR < 256 ? 256 : TPR;
    const int64_t n = (a.rows + RPB - 1) / RPB, most = 1 << 21;  // a grid's side: fewer than 2^32 threads
    const dim3 grid((unsigned)(n < most ? n : most), (unsigned)((n + most - 1) / most));
    hipLaunchKernelGGL((norm_kernel<TPR, NV, TAIL>), grid, dim3(THR), 0, st, a);
}
template <int TPR, int NV, bool TAIL>
void norm_launch(const NormBwdArgs& a, hipStream_t st) {
    constexpr int THR = TPR < 256 ? 256 : TPR;
    hipLaunchKernelGGL((norm_bwd_kernel<TPR, NV, TAIL>), dim3((unsigned)a.blocks), dim3(THR), TPR < 256 ? a.d * 4 : 0, st, a);
}

// Threads a row: as many as it has pieces up to a wavefront (16 and 32 for the
// narrow ones; no LDS exchange), then 256 or 1024, so that a row takes few
// registers of each. (Backward of 2^25 elements in bf16, in TB/s, with 64 threads of
// 4 pieces, 256 of 4 and of 8 / as here: d = 1536: 2.9 / 3.8, 8192: 2.7 / 3.8, 16384: 1.5 / 3.9.)
int row_threads(int n) { return n <= 16 ? 16 : n <= 32 ? 32 : n <= 128 ? 64 : n <= 512 ? 256 : 1024; }

template <bool TAIL, typename A>
hipError_t norm_dispatch(const A& a, hipStream_t st) {
    const int n = (a.d + VEC - 1) / VEC;
    switch (row_threads(n)) {
        case 16: norm_launch<16, 1, TAIL>(a, st); break;
        case 32: norm_launch<32, 1, TAIL>(a, st); break;
        case 64: n <= 64 ? norm_launch<64, 1, TAIL>(a, st) : norm_launch<64, 2, TAIL>(a, st); break;
        case 256: n <= 256 ? norm_launch<256, 1, TAIL>(a, st) : norm_launch<256, 2, TAIL>(a, st); break;
        default: n <= 1024 ? norm_launch<1024, 1, TAIL>(a, st) : norm_launch<1024, 2, TAIL>(a, st);
    }
    return hipGetLastError();
}
template <typename A>
hipError_t norm_any(const A& a, hipStream_t st) {
    return a.d % VEC ? norm_dispatch<true>(a, st) : norm_dispatch<false>(a, st);
}

}  // namespace

int64_t norm_bwd_blocks(int64_t rows, int d) {
    const int tpr = row_threads((d + VEC - 1) / VEC), rpb = tpr < 256 ? 256 / tpr : 1;
    const int64_t need = (rows + rpb - 1) / rpb, most = 256 * (tpr == 1024 ? 1 : 4);  // what the CUs hold at once
    return need < most ? need : most;
}

hipError_t launch_norm(const NormArgs& a, hipStream_t st) { return norm_any(a, st); }

hipError_t launch_norm_backward(NormBwdArgs a, hipStream_t st) {
    a.blocks = (int)norm_bwd_blocks(a.rows, a.d);
    hipError_t e = norm_any(a, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)((a.d + 15) / 16)), dim3(1024), 0, st, a.part, a.dgamma,
                       a.blocks, a.d);
    return hipGetLastError();
}

}  // namespace sdm
