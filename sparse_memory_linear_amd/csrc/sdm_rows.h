// sdm_rows.h -- device helpers of the state-space layer's kernels: pieces of rows in fp32 or
// bf16, and the activations.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {
namespace {

__device__ __forceinline__ float bf16_f(uint32_t u) { return __uint_as_float(u << 16); }
// nearest even, in one instruction; a NaN stays one
__device__ __forceinline__ uint32_t f_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 1 / (1 + e^-x): 0 and 1 at the ends
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * x));
}

// VEC elements of a row as they are stored: pieces of 4 or more elements aligned to their bytes (16 at most), or single ones
template <int VEC, bool BF16>
struct Piece {
    static constexpr int W = BF16 ? (VEC + 1) / 2 : VEC;
    uint32_t u[W];
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        const char* at = static_cast<const char*>(p) + e * (BF16 ? 2 : 4);
        if constexpr (W % 4 == 0) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const uint4 x = reinterpret_cast<const uint4*>(at)[i / 4];
                u[i] = x.x; u[i + 1] = x.y; u[i + 2] = x.z; u[i + 3] = x.w;
            }
        } else if constexpr (BF16 && VEC == 4) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            u[0] = x.x; u[1] = x.y;
        } else {
            static_assert(!BF16 || VEC == 1, "");
#pragma unroll
            for (int i = 0; i < W; ++i)
                if constexpr (BF16) u[i] = reinterpret_cast<const uint16_t*>(at)[i];
                else u[i] = reinterpret_cast<const uint32_t*>(at)[i];
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (BF16) return __uint_as_float(i & 1 ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
        else return __uint_as_float(u[i]);
    }
};
template <int VEC, bool BF16>
__device__ __forceinline__ void load_piece(const void* p, int64_t e, float (&v)[VEC]) {
    Piece<VEC, BF16> x;
    x.load(p, e);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = x[i];
}

template <int VEC, bool BF16>
__device__ __forceinline__ void store_piece(void* p, int64_t e, const float (&v)[VEC]) {
    if constexpr (BF16) {
        uint16_t* b = static_cast<uint16_t*>(p) + e;
        if constexpr (VEC % 4 == 0) {
            uint32_t u[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) u[i] = f_bf16(v[2 * i]) | f_bf16(v[2 * i + 1]) << 16;
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(b) = make_uint4(u[0], u[1], u[2], u[3]);
            else *reinterpret_cast<uint2*>(b) = make_uint2(u[0], u[1]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) b[i] = (uint16_t)f_bf16(v[i]);
        }
    } else {
        float* f = static_cast<float*>(p) + e;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(f + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = v[i];
        }
    }
}

// the value of another lane of the 16: quad permutes 0xB1 (lane ^ 1) and 0x4E (lane ^ 2), 0x141 (lane 7 - j of the half
// row), 0x140 (lane 15 - j), 0x128 (lane ^ 8)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}
// The sum over groups of N lanes (16, 32, 64), the same in all of them
template <int N>
__device__ __forceinline__ float lane_sum(float x) {
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    x += dpp<0x141>(x);
    x += dpp<0x140>(x);
    if constexpr (N >= 32) {
        const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    if constexpr (N >= 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    return x;
}

// out(i, the sum of column i of part [rows][cols], in 64 bits): 32 columns a workgroup, 32 groups of lanes
// each adding every 32nd row, then their sums in order. The order follows from the sizes alone.
template <typename Out>
__global__ __launch_bounds__(1024) void sum_columns_kernel(const float* part, int64_t rows, int64_t cols, Out out) {
    __shared__ double s[32][33];
    const int l = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + l;
    double x = 0.0;
    if (i < cols)
#pragma unroll 4
        for (int64_t r = g; r < rows; r += 32) x += part[r * cols + i];
    s[g][l] = x;
    __syncthreads();
    if (g == 0 && i < cols) {
        for (int k = 1; k < 32; ++k) x += s[k][l];
        out(i, (float)x);
    }
}
template <typename Out>
hipError_t sum_columns(const float* part, int64_t rows, int64_t cols, const Out& out, hipStream_t st) {
    hipLaunchKernelGGL(sum_columns_kernel<Out>, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, st, part, rows, cols, out);
    return hipGetLastError();
}

}  // namespace
}  // namespace sdm
