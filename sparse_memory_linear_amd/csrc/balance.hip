// balance.hip -- slot counts and balance loss of an addressing result, on gfx950.
//   count[h,i] = selections of slot i by head h over the kept tokens (n of them)
//   mass[h,i]  = the sum of their weights
//   loss[h]    = N sum_i (count / (n K)) (mass / n)       (1 when all is even)
//   dwt        = dloss[h] N / n * count[idx] / (n K), 0 at tokens left out
//
// Weights are added as whole numbers (fixed point with 2^shift to one, 64
// bits), so the sums do not depend on the order in which they arrive. The shift
// leaves room for as many weights of magnitude 2 as a head has selections. A
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
//
// Measured: 16.8 M selections (4 x 8 x 8192 tokens of 64), 65536 slots, forward and
// backward 116 us: adding 59 (134 MB, 28 us at a copy's 4.75 TB/s; bound by the vector
// instructions that look at every selection once per range, 5 times here), tables and loss 13,
// backward 37 (134 MB). 64-bit atomics in memory in place of the tables in LDS took 2.0 ms in
// all. Dealing the slots to the ranges in turn, which evens out skewed use, took as long.
#include "sdm_buffer.h"
#include "sdm_internal.h"

namespace sdm {
namespace {

constexpr int RANGE = 13312;   // slots a workgroup: 12 bytes each, 156 KiB of LDS
constexpr int ADD_THREADS = 1024;
constexpr int MERGE_SLOTS = 512;
constexpr int64_t MOST = 1 << 23;  // tokens walked at a time: MOST K (2^40 / K + 1) < 2^64

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
    const int64_t h = s % a.H, share = s / a.H;  // s = share * H + h
    const uint32_t lo = (uint32_t)r * a.range, len = min((uint32_t)a.range, (uint32_t)a.N - lo);
    for (uint32_t i = tid; i < len; i += ADD_THREADS) { mass[i] = 0; count[i] = 0; }
    if (tid == 0) { bad = 0; kept = 0; }
    __syncthreads();
    const double base = fix_base(a.shift);
    const uint64_t kdiv = ((1ull << 40) / (uint64_t)a.K) + 1;  // e / K = e kdiv >> 40 for e < MOST K, K <= 256
    auto take = [&](int32_t slot, float w) {
        const uint32_t i = (uint32_t)slot - lo;
        if (i < len) {
            atomicAdd(&count[i], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&mass[i]),
                      (unsigned long long)__double_as_longlong((double)w + base));
        }
    };
    // (a weight that is NaN or out of range spoils its head's sums; the first range looks)
    const int64_t ntok = a.B * a.T;
    const int64_t u0 = share * a.share, u1 = u0 + a.share < ntok ? u0 + a.share : ntok;
    for (int64_t u = u0; u < u1;) {  // one sequence's tokens at a time: contiguous selections
        const int64_t b = u / a.T, t = u - b * a.T;
        const int64_t m = min(min(a.T - t, u1 - u), MOST);
        const int64_t at = ((b * a.H + h) * a.T + t) * a.K;
        const uint8_t* keep = a.mask ? a.mask + b * a.T + t : nullptr;
        const uint32_t n = (uint32_t)(m * a.K);  // < 2^31 (host)
        auto on = [&](uint32_t e) { return !keep || keep[((uint64_t)e * kdiv) >> 40] != 0; };
        // a batch's loads are all issued before its first selection is taken
        constexpr int NB = 4, W = VEC ? 4 : 1;  // VEC: K a multiple of 4, pieces of 16 bytes
        for (uint32_t e0 = tid; e0 < n / W; e0 += NB * ADD_THREADS) {
            int32_t i[NB][W];
            float w[NB][W];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t e = e0 + k * ADD_THREADS;
                const bool in = e < n / W;
                const bool kept = in && on(e * W);  // (loaded beside the selections, not in front of them)
                if constexpr (VEC) {
                    int4 x = make_int4(-1, -1, -1, -1);
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (in) {
                        x = reinterpret_cast<const int4*>(a.idx + at)[e];
                        y = reinterpret_cast<const float4*>(a.wt + at)[e];
                    }
                    if (!kept) x = make_int4(-1, -1, -1, -1);
                    i[k][0] = x.x; i[k][1] = x.y; i[k][2] = x.z; i[k][3] = x.w;
                    w[k][0] = y.x; w[k][1] = y.y; w[k][2] = y.z; w[k][3] = y.w;
                } else {
                    i[k][0] = in ? a.idx[at + e] : -1;
                    if (!kept) i[k][0] = -1;
                    w[k][0] = in ? a.wt[at + e] : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int j = 0; j < W; ++j) take(i[k][j], w[k][j]);
            if (r == 0) {
                bool b = false;
#pragma unroll
                for (int k = 0; k < NB; ++k)
#pragma unroll
                    for (int j = 0; j < W; ++j) b |= !(fabsf(w[k][j]) <= 2.f) && (uint32_t)i[k][j] < (uint32_t)a.N;
                if (b) bad = 1;
            }
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
        if (r == 0) a.bad[s] = bad;
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
    for (int64_t i = threadIdx.x; i < a.nshare; i += 256)
        if (a.bad[i * a.H + h]) any = 1;
    __syncthreads();
    const double unit = ldexp(1.0, -a.shift);
    const bool bad = any != 0;
    double sum = 0.0;
    const int64_t end = (int64_t)(blk + 1) * MERGE_SLOTS < a.N ? (int64_t)(blk + 1) * MERGE_SLOTS : a.N;
    for (int64_t i = (int64_t)blk * MERGE_SLOTS + threadIdx.x; i < end; i += 256) {
        int64_t f = 0;
        int32_t c = 0;
#pragma unroll 8
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

// A workgroup per piece of one head's selections. TABLE: the head's counts sit in
// LDS, 16 bits each (65535: that many or more, taken from memory), so that the
// gather does not go to the L2, a line a selection; else they are gathered there.
template <bool VEC, bool TABLE>
__global__ __launch_bounds__(TABLE ? 1024 : 256) void balance_bwd_kernel(BalanceBwdArgs a) {
    constexpr int THR = TABLE ? 1024 : 256;
    extern __shared__ __align__(16) uint16_t table[];
    const int64_t h = blockIdx.x % a.H, piece = blockIdx.x / a.H;
    const double n = (double)*a.tokens;
    const float c = n > 0.0 ? (float)((double)a.dloss[h] * ((double)a.N / (n * n * (double)a.K))) : 0.f;
    const int32_t* counts = a.counts + h * a.N;
    const uint32_t N = (uint32_t)a.N;
    if constexpr (TABLE) {
        for (uint32_t i = threadIdx.x; i < N; i += THR) table[i] = (uint16_t)min(counts[i], 65535);
        __syncthreads();
    }
    const uint64_t kdiv = ((1ull << 40) / (uint64_t)a.K) + 1;  // e / K = e kdiv >> 40 for e < MOST K, K <= 256
    auto grad = [&](int32_t slot) {
        if ((uint32_t)slot >= N) return 0.f;
        int k;
        if constexpr (TABLE) {
            k = table[slot];
            if (k == 65535) k = counts[slot];
        } else {
            k = counts[slot];
        }
        return c * (float)k;
    };
    const int64_t ntok = a.B * a.T;
    const int64_t u0 = piece * a.piece, u1 = u0 + a.piece < ntok ? u0 + a.piece : ntok;
    for (int64_t u = u0; u < u1;) {  // one sequence's tokens at a time: contiguous selections
        const int64_t b = u / a.T, t = u - b * a.T;
        const int64_t m = min(min(a.T - t, u1 - u), MOST);
        const int64_t at = ((b * a.H + h) * a.T + t) * a.K;
        const uint8_t* keep = a.mask ? a.mask + b * a.T + t : nullptr;
        const uint32_t e1 = (uint32_t)(m * a.K);
        auto on = [&](uint32_t e) { return !keep || keep[((uint64_t)e * kdiv) >> 40] != 0; };
        if constexpr (VEC) {
            const int4* ip = reinterpret_cast<const int4*>(a.idx + at);
            float4* op = reinterpret_cast<float4*>(a.dwt + at);
#pragma unroll 4
            for (uint32_t e = threadIdx.x; e < e1 / 4; e += THR) {
                const int4 i = ip[e];
                op[e] = on(e * 4) ? make_float4(grad(i.x), grad(i.y), grad(i.z), grad(i.w)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else {
            for (uint32_t e = threadIdx.x; e < e1; e += THR) a.dwt[at + e] = on(e) ? grad(a.idx[at + e]) : 0.f;
        }
        u += m;
    }
}

template <bool VEC>
void balance_bwd_launch(BalanceBwdArgs a, hipStream_t st) {
    // The table pays where a workgroup per CU has at least half as many selections as
    // slots to load, and holds up to 80 K slots (16.8 M selections, 65536 slots, as
    // many a workgroup as slots: 37 us, and 65 without).
    const int64_t sel = a.B * a.T * a.K, wgs = a.H < 256 ? 256 / a.H : 1;
    const bool table = a.N <= 80 * 1024 && sel / wgs >= a.N / 2;
    a.piece = table ? (a.B * a.T + wgs - 1) / wgs : (BALANCE_PIECE + a.K - 1) / a.K;
    const dim3 grid((unsigned)(a.H * ((a.B * a.T + a.piece - 1) / a.piece)));
    if (table) hipLaunchKernelGGL((balance_bwd_kernel<VEC, true>), grid, dim3(1024), (a.N * 2 + 15) / 16 * 16, st, a);
    else hipLaunchKernelGGL((balance_bwd_kernel<VEC, false>), grid, dim3(256), 0, st, a);
}

// Shares of the tokens: a workgroup per CU (an LDS range fills one), but no
// share with fewer selections than a quarter of the slots: a share's table is
// written and read once more (504 K selections over 262144 slots: 48 us with 7
// shares, 80 with 12).
struct BalanceLayout {
    int64_t nrange, range, nshare, share, nblk, fixed, counts, bad, kept, bytes;
};
BalanceLayout balance_layout(int64_t B, int64_t H, int64_t T, int64_t K, int64_t N) {
    BalanceLayout y{};
    y.nrange = (N + RANGE - 1) / RANGE;
    y.range = (N + y.nrange - 1) / y.nrange;
    const int64_t tok = B * T;
    int64_t n = 256 / (H * y.nrange);
    const int64_t most = tok * K / (N / 4 + 1);
    if (n > most) n = most;
    if (n < 1) n = 1;
    y.share = (tok + n - 1) / n;
    y.nshare = y.share > 0 ? (tok + y.share - 1) / y.share : 1;
    y.nblk = (N + MERGE_SLOTS - 1) / MERGE_SLOTS;
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    y.fixed = up(y.nshare * H * N * 8);
    y.counts = up(y.nshare * H * N * 4);
    y.bad = up(y.nshare * H * 4);
    y.kept = up(y.nshare * 4);
    y.bytes = y.fixed + y.counts + y.bad + y.kept + H * y.nblk * 8;
    return y;
}

}  // namespace

int64_t balance_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t K, int64_t N) {
    return balance_layout(B, H, T, K, N).bytes;
}

hipError_t launch_balance(BalanceArgs a, hipStream_t st) {
    const BalanceLayout y = balance_layout(a.B, a.H, a.T, a.K, a.N);
    char* p = static_cast<char*>(a.workspace);
    a.fixed = reinterpret_cast<int64_t*>(p);
    a.part_counts = reinterpret_cast<int32_t*>(p += y.fixed);
    a.bad = reinterpret_cast<int32_t*>(p += y.counts);
    a.kept = reinterpret_cast<int32_t*>(p += y.bad);
    a.part = reinterpret_cast<double*>(p += y.kept);
    a.nrange = (int)y.nrange; a.range = (int)y.range; a.nshare = y.nshare; a.share = y.share; a.nblk = (int)y.nblk;
    int bits = 0;
    while ((int64_t)1 << bits < a.B * a.T * a.K) ++bits;
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
    if (a.K % 4 == 0) balance_bwd_launch<true>(a, st);
    else balance_bwd_launch<false>(a, st);
    return hipGetLastError();
}

}  // namespace sdm
