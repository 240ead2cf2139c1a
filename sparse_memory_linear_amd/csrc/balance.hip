// balance.hip -- slot counts and balance loss of an addressing result, on gfx950.
//   count[h,i] = selections of slot i by head h over the kept tokens (n of them)
//   mass[h,i]  = the sum of their weights
//   loss[h]    = N sum_i (count / (n K)) (mass / n)       (1 when all is even)
//   dwt        = dloss[h] N / n * count[idx] / (n K), 0 at tokens left out
//
// Weights are added as whole numbers (fixed point with 2^shift to one, 64
// bits), so the sums do not depend on the order in which they arrive. The shift
// leaves room for as many weights of magnitude 2 as the call has entries.
#include "sdm_internal.h"

namespace sdm {
namespace {

__global__ __launch_bounds__(256) void balance_clear_kernel(uint32_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// kept tokens, by one workgroup
__global__ __launch_bounds__(1024) void balance_tokens_kernel(const uint8_t* mask, int64_t n, int32_t* tokens) {
    __shared__ int part[16];
    int x = 0;
    if (mask)
        for (int64_t i = threadIdx.x; i < n; i += 1024) x += mask[i] != 0;
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    if (threadIdx.x) return;
    x = 0;
    for (int i = 0; i < 16; ++i) x += part[i];
    *tokens = mask ? x : (int32_t)n;
}

__global__ __launch_bounds__(256) void balance_add_kernel(BalanceArgs a) {
    const int64_t n = a.B * a.H * a.T * a.K;
    const float one = ldexpf(1.f, a.shift);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t tok = i / a.K, bh = tok / a.T, t = tok - bh * a.T, b = bh / a.H, h = bh - b * a.H;
        if (a.mask && !a.mask[b * a.T + t]) continue;
        const uint32_t slot = (uint32_t)a.idx[i];
        if (slot >= (uint32_t)a.N) continue;
        const float w = a.wt[i];
        atomicAdd(&a.counts[h * a.N + slot], 1);
        if (!(fabsf(w) <= 2.f)) atomicOr(&a.bad[h], 1);
        else atomicAdd(reinterpret_cast<unsigned long long*>(&a.fixed[h * a.N + slot]), (unsigned long long)llrintf(w * one));
    }
}

// mass in fp32, and per block of slots the sum of count * mass in fp64
__global__ __launch_bounds__(256) void balance_mass_kernel(BalanceArgs a) {
    __shared__ double part[4];
    const int64_t h = blockIdx.x / a.nblk;
    const int blk = (int)(blockIdx.x % a.nblk);
    const double unit = ldexp(1.0, -a.shift);
    const bool bad = a.bad[h] != 0;
    double sum = 0.0;
    const int64_t end = (int64_t)(blk + 1) * a.per < a.N ? (int64_t)(blk + 1) * a.per : a.N;
    for (int64_t i = (int64_t)blk * a.per + threadIdx.x; i < end; i += 256) {
        const double m = (double)a.fixed[h * a.N + i] * unit;
        sum += (double)a.counts[h * a.N + i] * m;
        a.mass[h * a.N + i] = bad ? __int_as_float(0x7FC00000) : (float)m;
    }
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.part[blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(64) void balance_loss_kernel(BalanceArgs a) {
    const int64_t h = blockIdx.x;
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.nblk; i += 64) sum += a.part[h * a.nblk + i];
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if (threadIdx.x) return;
    const double n = (double)*a.tokens;
    const float l = n > 0.0 ? (float)((double)a.N * sum / (n * (double)a.K) / n) : 0.f;
    a.loss[h] = a.bad[h] ? __int_as_float(0x7FC00000) : l;
}

__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
    const int64_t n = a.B * a.H * a.T * a.K;
    const double tok_n = (double)*a.tokens;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t tok = i / a.K, bh = tok / a.T, t = tok - bh * a.T, b = bh / a.H, h = bh - b * a.H;
        const uint32_t slot = (uint32_t)a.idx[i];
        float d = 0.f;
        if ((!a.mask || a.mask[b * a.T + t]) && slot < (uint32_t)a.N)
            d = (float)((double)a.dloss[h] * ((double)a.N / (tok_n * tok_n * (double)a.K))) * (float)a.counts[h * a.N + slot];
        a.dwt[i] = d;
    }
}

}  // namespace

int64_t balance_blocks(int64_t N) { return (N + 4095) / 4096; }
int64_t balance_workspace_bytes(int64_t H, int64_t N) {
    return H * N * 8 + (H * 4 + 15) / 16 * 16 + H * balance_blocks(N) * 8;
}

hipError_t launch_balance(BalanceArgs a, hipStream_t st) {
    const int64_t n = a.B * a.H * a.T * a.K;
    char* ws = static_cast<char*>(a.workspace);
    a.fixed = reinterpret_cast<int64_t*>(ws);
    a.bad = reinterpret_cast<int32_t*>(ws + a.H * a.N * 8);
    a.part = reinterpret_cast<double*>(ws + a.H * a.N * 8 + (a.H * 4 + 15) / 16 * 16);
    a.nblk = (int)balance_blocks(a.N);
    a.per = 4096;
    int bits = 0;
    while ((int64_t)1 << bits < n) ++bits;
    a.shift = 61 - bits < 40 ? 61 - bits : 40;
    auto blocks = [](int64_t m) { return dim3((unsigned)((m + 255) / 256 < 8192 ? (m + 255) / 256 : 8192)); };
    const int64_t own = a.H * a.N * 2 + a.H;  // words of `fixed` and `bad`
    hipLaunchKernelGGL(balance_clear_kernel, blocks(own), dim3(256), 0, st, reinterpret_cast<uint32_t*>(ws), own);
    hipLaunchKernelGGL(balance_clear_kernel, blocks(a.H * a.N), dim3(256), 0, st,
                       reinterpret_cast<uint32_t*>(a.counts), a.H * a.N);
    hipLaunchKernelGGL(balance_tokens_kernel, dim3(1), dim3(1024), 0, st, a.mask, a.B * a.T, a.tokens);
    if (n > 0) hipLaunchKernelGGL(balance_add_kernel, blocks(n), dim3(256), 0, st, a);
    hipLaunchKernelGGL(balance_mass_kernel, dim3((unsigned)(a.H * a.nblk)), dim3(256), 0, st, a);
    hipLaunchKernelGGL(balance_loss_kernel, dim3((unsigned)a.H), dim3(64), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceBwdArgs& a, hipStream_t st) {
    const int64_t n = a.B * a.H * a.T * a.K, b = (n + 255) / 256;
    hipLaunchKernelGGL(balance_bwd_kernel, dim3((unsigned)(b < 16384 ? b : 16384)), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace sdm
