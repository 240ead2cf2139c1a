// balance.hip -- slot counts and balance loss of an addressing result, on gfx950.
//   count[h,i] = selections of slot i by head h over the kept tokens (n of them)
//   mass[h,i]  = the sum of their weights
//   loss[h]    = N sum_i (count / (n K)) (mass / n)       (1 when all is even)
//   dwt        = dloss[h] N / n * count[idx] / (n K), 0 at tokens left out
//
// Weights are added as whole numbers (fixed point with 2^shift to one, 64
// bits), so the sums do not depend on the order in which they arrive. The shift
// leaves room for as many weights of magnitude 2 as the call has entries. A
// weight becomes one by an fp64 addition: w + 1.5 2^(52 - shift) holds the
// rounded w 2^shift in its low bits, so the raw bits are added, and the constant's
// are taken off count times at the end (modulo 2^64).
//
// balance_add_kernel: a workgroup holds a range of one head's slots in LDS (12
// bytes a slot, at most RANGE slots) and reads all selections of its share of the
// tokens, taking those that fall into its range; the ranges of one share run on
// one XCD at about the same time, so all but the first read them from its L2.
// Shares split the tokens until there is a workgroup per CU. The second kernel
// adds the shares' tables.
#include "sdm_buffer.h"
#include "sdm_internal.h"

namespace sdm {
namespace {

constexpr int RANGE = 13312;   // slots a workgroup: 12 bytes each, 156 KiB of LDS
constexpr int ADD_THREADS = 1024;
constexpr int MERGE_SLOTS = 2048;

// fp64 whose unit in the last place is 2^-shift
__device__ __forceinline__ double fix_base(int shift) { return ldexp(1.5, 52 - shift); }

template <bool VEC>
__global__ __launch_bounds__(ADD_THREADS) void balance_add_kernel(BalanceArgs a) {
    extern __shared__ __align__(16) char lds[];
    uint64_t* mass = reinterpret_cast<uint64_t*>(lds);
    uint32_t* count = reinterpret_cast<uint32_t*>(lds + (int64_t)a.range * 8);
    __shared__ int bad, kept;
    const int tid = threadIdx.x;
    int64_t s;
    int r;
    block_unit((int)blockIdx.x, a.H * a.nshare, a.nrange, s, r);
    if (s >= a.H * a.nshare) return;
    const int64_t h = s % a.H, share = s / a.H;
    const uint32_t lo = (uint32_t)r * a.range, len = min((uint32_t)a.range, (uint32_t)a.N - lo);
    for (uint32_t i = tid; i < len; i += ADD_THREADS) { mass[i] = 0; count[i] = 0; }
    if (tid == 0) { bad = 0; kept = 0; }
    __syncthreads();
    const double base = fix_base(a.shift);
    const uint64_t kdiv = ((1ull << 40) / (uint64_t)a.K) + 1;  // e / K = e kdiv >> 40 for e < 2^32, K <= 256
    auto take = [&](int32_t slot, float w) {
        const uint32_t i = (uint32_t)slot - lo;
        if (i < len) {
            atomicAdd(&count[i], 1u);
            if (fabsf(w) <= 2.f) {
                atomicAdd(reinterpret_cast<unsigned long long*>(&mass[i]),
                          (unsigned long long)__double_as_longlong((double)w + base));
            } else {  // NaN or out of range: the constant alone
                atomicAdd(reinterpret_cast<unsigned long long*>(&mass[i]), (unsigned long long)__double_as_longlong(base));
                bad = 1;
            }
        }
    };
    const int64_t ntok = a.B * a.T;
    const int64_t u0 = share * a.share, u1 = u0 + a.share < ntok ? u0 + a.share : ntok;
    for (int64_t u = u0; u < u1;) {  // one sequence's tokens at a time: contiguous selections
        const int64_t b = u / a.T, t = u - b * a.T;
        const int64_t m = a.T - t < u1 - u ? a.T - t : u1 - u;
        const int64_t at = ((b * a.H + h) * a.T + t) * a.K;
        const uint8_t* keep = a.mask ? a.mask + b * a.T + t : nullptr;
        const uint32_t n = (uint32_t)(m * a.K);
        auto on = [&](uint32_t e) { return !keep || keep[((uint64_t)e * kdiv) >> 40] != 0; };
        if constexpr (VEC) {  // K a multiple of 4: a token's selections in pieces of 16 bytes
            const int4* ip = reinterpret_cast<const int4*>(a.idx + at);
            const float4* wp = reinterpret_cast<const float4*>(a.wt + at);
#pragma unroll 4
            for (uint32_t e = tid; e < n / 4; e += ADD_THREADS) {
                if (!on(e * 4)) continue;
                const int4 i = ip[e];
                const float4 w = wp[e];
                take(i.x, w.x); take(i.y, w.y); take(i.z, w.z); take(i.w, w.w);
            }
        } else {
#pragma unroll 4
            for (uint32_t e = tid; e < n; e += ADD_THREADS)
                if (on(e)) take(a.idx[at + e], a.wt[at + e]);
        }
        if (h == 0 && r == 0 && keep) {
            int c = 0;
            for (int64_t i = tid; i < m; i += ADD_THREADS) c += keep[i] != 0;
            if (c) atomicAdd(&kept, c);
        }
        u += m;
    }
    __syncthreads();
    const uint64_t off = (uint64_t)__double_as_longlong(base);
    const int64_t o = (share * a.H + h) * a.N + lo;
    for (uint32_t i = tid; i < len; i += ADD_THREADS) {
        a.fixed[o + i] = (int64_t)(mass[i] - (uint64_t)count[i] * off);
        a.part_counts[o + i] = (int32_t)count[i];
    }
    if (tid == 0) {
        a.bad[s * a.nrange + r] = bad;
        if (h == 0 && r == 0) a.kept[share] = a.mask ? kept : (int32_t)(u1 - u0);
    }
}

// The shares' tables added up; per block of slots, the sum of count * mass in fp64
__global__ __launch_bounds__(256) void balance_mass_kernel(BalanceArgs a) {
    __shared__ double part[4];
    __shared__ int any;
    const int64_t h = blockIdx.x / a.nblk;
    const int blk = (int)(blockIdx.x % a.nblk);
    if (threadIdx.x == 0) any = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.nshare * (int64_t)a.nrange; i += 256)
        if (a.bad[(i / a.nrange * a.H + h) * a.nrange + i % a.nrange]) any = 1;
    __syncthreads();
    const double unit = ldexp(1.0, -a.shift);
    const bool bad = any != 0;
    double sum = 0.0;
    const int64_t end = (int64_t)(blk + 1) * MERGE_SLOTS < a.N ? (int64_t)(blk + 1) * MERGE_SLOTS : a.N;
    for (int64_t i = (int64_t)blk * MERGE_SLOTS + threadIdx.x; i < end; i += 256) {
        int64_t f = 0;
        int32_t c = 0;
        for (int64_t s = 0; s < a.nshare; ++s) {
            f += a.fixed[(s * a.H + h) * a.N + i];
            c += a.part_counts[(s * a.H + h) * a.N + i];
        }
        const double m = (double)f * unit;
        sum += (double)c * m;
        a.counts[h * a.N + i] = c;
        a.mass[h * a.N + i] = bad ? __int_as_float(0x7FC00000) : (float)m;
    }
    for (int m = 1; m < 64; m <<= 1) sum += __shfl_xor(sum, m);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0)
        a.part[blockIdx.x] = bad ? __longlong_as_double(0x7FF8000000000000ll) : (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(64) void balance_loss_kernel(BalanceArgs a) {
    const int64_t h = blockIdx.x;
    double sum = 0.0;
    int tok = 0;
    for (int i = threadIdx.x; i < a.nblk; i += 64) sum += a.part[h * a.nblk + i];
    for (int64_t i = threadIdx.x; i < a.nshare; i += 64) tok += a.kept[i];
    for (int m = 1; m < 64; m <<= 1) {
        sum += __shfl_xor(sum, m);
        tok += __shfl_xor(tok, m);
    }
    if (threadIdx.x) return;
    const double n = (double)tok;
    a.loss[h] = tok > 0 ? (float)((double)a.N * sum / (n * (double)a.K) / n) : 0.f;
    if (h == 0) *a.tokens = tok;
}

// A workgroup per piece of one (b, h)'s selections; the head's counts are
// gathered from the L2.
template <bool VEC>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceBwdArgs a) {
    const int64_t bh = blockIdx.x / a.pieces, piece = blockIdx.x % a.pieces;
    const int64_t b = bh / a.H, h = bh - b * a.H, run = a.T * a.K;
    const double n = (double)*a.tokens;
    const float c = n > 0.0 ? (float)((double)a.dloss[h] * ((double)a.N / (n * n * (double)a.K))) : 0.f;
    const int32_t* counts = a.counts + h * a.N;
    const uint32_t N = (uint32_t)a.N;
    const uint8_t* keep = a.mask ? a.mask + b * a.T : nullptr;
    const uint64_t kdiv = ((1ull << 40) / (uint64_t)a.K) + 1;  // e / K = e kdiv >> 40 for e < 2^32, K <= 256
    auto on = [&](uint32_t e) { return !keep || keep[((uint64_t)e * kdiv) >> 40] != 0; };
    auto grad = [&](int32_t slot) { return (uint32_t)slot < N ? c * (float)counts[slot] : 0.f; };
    const int64_t e0 = piece * BALANCE_PIECE, e1 = e0 + BALANCE_PIECE < run ? e0 + BALANCE_PIECE : run;
    if constexpr (VEC) {
        const int4* ip = reinterpret_cast<const int4*>(a.idx + bh * run);
        float4* op = reinterpret_cast<float4*>(a.dwt + bh * run);
#pragma unroll 4
        for (int64_t e = e0 / 4 + threadIdx.x; e < e1 / 4; e += 256) {
            const int4 i = ip[e];
            op[e] = on((uint32_t)e * 4) ? make_float4(grad(i.x), grad(i.y), grad(i.z), grad(i.w)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    } else {
        for (int64_t e = e0 + threadIdx.x; e < e1; e += 256)
            a.dwt[bh * run + e] = on((uint32_t)e) ? grad(a.idx[bh * run + e]) : 0.f;
    }
}

// Shares of the tokens: a workgroup per CU (an LDS range fills one), but no
// share below 256 tokens, whose tables would cost more than its selections.
struct BalanceLayout {
    int64_t nrange, range, nshare, share, nblk, fixed, counts, bad, kept, bytes;
};
BalanceLayout balance_layout(int64_t B, int64_t H, int64_t T, int64_t N) {
    BalanceLayout y{};
    y.nrange = (N + RANGE - 1) / RANGE;
    y.range = (N + y.nrange - 1) / y.nrange;
    const int64_t tok = B * T;
    int64_t n = 256 / (H * y.nrange);
    if (n > (tok + 255) / 256) n = (tok + 255) / 256;
    if (n < 1) n = 1;
    y.share = (tok + n - 1) / n;
    y.nshare = y.share > 0 ? (tok + y.share - 1) / y.share : 1;
    y.nblk = (N + MERGE_SLOTS - 1) / MERGE_SLOTS;
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    y.fixed = up(y.nshare * H * N * 8);
    y.counts = up(y.nshare * H * N * 4);
    y.bad = up(y.nshare * H * y.nrange * 4);
    y.kept = up(y.nshare * 4);
    y.bytes = y.fixed + y.counts + y.bad + y.kept + H * y.nblk * 8;
    return y;
}

}  // namespace

int64_t balance_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t N) { return balance_layout(B, H, T, N).bytes; }

hipError_t launch_balance(BalanceArgs a, hipStream_t st) {
    const BalanceLayout y = balance_layout(a.B, a.H, a.T, a.N);
    char* p = static_cast<char*>(a.workspace);
    a.fixed = reinterpret_cast<int64_t*>(p);
    a.part_counts = reinterpret_cast<int32_t*>(p += y.fixed);
    a.bad = reinterpret_cast<int32_t*>(p += y.counts);
    a.kept = reinterpret_cast<int32_t*>(p += y.bad);
    a.part = reinterpret_cast<double*>(p += y.kept);
    a.nrange = (int)y.nrange; a.range = (int)y.range; a.nshare = y.nshare; a.share = y.share; a.nblk = (int)y.nblk;
    int bits = 0;
    while ((int64_t)1 << bits < a.B * a.H * a.T * a.K) ++bits;
    a.shift = 61 - bits < 40 ? 61 - bits : 40;
    const dim3 grid((unsigned)unit_grid(a.H * a.nshare, a.nrange));
    const int bytes = a.range * 12;
    if (a.K % 4 == 0) hipLaunchKernelGGL(balance_add_kernel<true>, grid, dim3(ADD_THREADS), bytes, st, a);
    else hipLaunchKernelGGL(balance_add_kernel<false>, grid, dim3(ADD_THREADS), bytes, st, a);
    hipLaunchKernelGGL(balance_mass_kernel, dim3((unsigned)(a.H * a.nblk)), dim3(256), 0, st, a);
    hipLaunchKernelGGL(balance_loss_kernel, dim3((unsigned)a.H), dim3(64), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_balance_backward(BalanceBwdArgs a, hipStream_t st) {
    a.pieces = (a.T * a.K + BALANCE_PIECE - 1) / BALANCE_PIECE;
    const dim3 grid((unsigned)(a.B * a.H * a.pieces));
    if (a.K % 4 == 0) hipLaunchKernelGGL(balance_bwd_kernel<true>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(balance_bwd_kernel<false>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace sdm
