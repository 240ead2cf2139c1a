// Internal launch interface between the C ABI (sdm_api.hip) and the kernels.
// Not installed, not part of the ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sdm {

struct AddressArgs {
    const void* q[2];        // per branch: [B,H,T,2,dh]
    const void* K[2];        // per branch: [H,2,n,dh]
    int32_t* idx[2];         // [B,H,T,k]
    float* wt[2];
    float* score[2];         // optional
    int k[2];
    float* half_out;         // debug: [B,H,T,2,n]; when set only half-scores are written
    int64_t B, H, T;
    int n, dh;
    int nbranch;             // 1 or 2
    bool bf16;
    bool idw;                // inverse-distance half-scores instead of dot products
};
hipError_t launch_address(const AddressArgs& a, hipStream_t st);

// The output step fused into the scan's last pass (partial sums of the row
// partitions -> y -> RMS-Norm and output gate -> o): see sdm_scan_forward_gated.
struct GateArgs {
    const float* gamma;      // [H,dv]
    const void* g;           // [B,H,T,dv] gate pre-activation
    float* o;                // [B,H,T,dv]
    float eps;
    int64_t H;
    bool g_bf16;
};

struct ScanArgs {
    const int32_t* idx_w; const float* wt_w; int W;
    const int32_t* idx_r; const float* wt_r; int R;
    const float* alpha; const float* beta;
    const void* v; bool v_bf16;
    void* M; bool m_bf16;    // table elements: fp32, or bfloat16 (no pre-images then)
    float* y;
    int64_t NS;              // B*H streams
    int64_t T, N;
    int dv;
    int form;                // 0 = per-slot Eq. (4), 1 = Fig. 2 shared residual
    void* workspace;
    float* snap;             // optional [NS][T][W][dv]: pre-image of every write (training forward)
    int64_t max_tokens = 0;  // > 0: tokens per launch chunk at most this (a bounded workspace)
    // optional: the output step; where the scan sums row-partition partials it
    // runs in that pass (y is then stored only if y != nullptr), else the caller
    // runs the output gate on y
    const GateArgs* gate = nullptr;
};
// Whether launch_scan with a.gate set fuses the output step for these sizes
// (else y is stored and the caller applies the gate).
bool scan_fuses_gate(int64_t NS, int64_t T, int W, int R, int dv, bool m_bf16, int form);
// Chooses the kernel instance; returns false if no instance covers (W, R, dv).
bool scan_geometry(int64_t NS, int W, int R, int dv, bool m_bf16, int* slab, int* rec_bytes);
int64_t scan_workspace_bytes(int64_t NS, int64_t T, int W, int R, int dv);
// The most tokens per launch chunk (at most T) whose workspace fits in `bytes`
// for this table dtype and form; T itself when the call takes the short-call
// form (no workspace); 0 when not even one token fits.
int64_t scan_tokens_within(int64_t NS, int64_t T, int W, int R, int dv, bool m_bf16, int form, int64_t bytes);
hipError_t launch_scan(const ScanArgs& a, hipStream_t st);

struct BwdArgs {
    const int32_t* idx_w; const float* wt_w; int W;
    const int32_t* idx_r; const float* wt_r; int R;
    const float* alpha; const float* beta;
    const void* v; bool v_bf16;
    const float* snap;       // [NS][T][W][dv] from the training forward
    const float* dy;         // [NS][T][dv]
    float* M;                // in: state after token T-1; out: before token 0 (restored)
    float* dM;               // in: dL/dM after token T-1; out: dL/dM before token 0
    float* dv_out;           // [NS][T][dv]
    float* dalpha; float* dbeta;   // [NS][T]
    float* dwt_w; float* dwt_r;    // [NS][T][W], [NS][T][R]
    int64_t NS, T, N;
    int dv;
    int form;
    void* workspace;
};
int64_t scan_backward_workspace_bytes(int64_t NS, int64_t T, int W, int R, int dv);
bool scan_backward_geometry(int64_t NS, int W, int R, int dv);
hipError_t launch_scan_backward(const BwdArgs& a, hipStream_t st);
hipError_t launch_state_init_backward(const float* dM, float* dM0, int64_t B, int64_t per_seq, hipStream_t st);

hipError_t launch_state_init(const float* M0, void* M, bool m_bf16, int64_t B, int64_t per_seq, hipStream_t st);

struct GatesArgs {
    const void* x;           // [B,T,d]
    const void* Wa;          // [H,d]
    const void* Wb;          // [H,d]
    const float* bdt;        // [H]
    const float* A;          // [H]
    float* alpha; float* beta;  // [B,H,T]
    int64_t B, T;
    int d, H;
    bool bf16;
};
hipError_t launch_gates(const GatesArgs& a, hipStream_t st);

struct OutGateArgs {
    const float* y;          // [B,H,T,dv]
    const float* gamma;      // [H,dv]
    const void* g;           // [B,H,T,dv]
    float* o;                // [B,H,T,dv]
    float eps;
    int64_t rows, T, H;      // rows = B*H*T
    int dv, lg;
    bool g_bf16;
};
hipError_t launch_output_gate(OutGateArgs a, hipStream_t st);

// Lanes per row of the output step: a power of two covering the row's 16-byte
// pieces, at most 64 (the same in the plain and the fused kernel, so both add
// the squares in the same order).
__host__ __device__ inline int output_gate_lanes(int dv) {
    int lg = 1;
    while (lg < 64 && lg < dv / 4) lg <<= 1;
    return lg;
}
// The fused form holds a lane's pieces in registers: at most this many.
constexpr int GATE_FUSED_PIECES = 4;
// The partial sums of P row partitions of one launch chunk (Tc of TS tokens
// from t0) -> y (if y != nullptr) and the output step -> o.
struct YGateArgs {
    const float* yp;         // [P][NS][Tc][dv]
    float* y;                // [NS][TS][dv] or nullptr
    GateArgs gate;
    int P;
    int64_t NS, Tc, TS, t0;
    int dv;
};
hipError_t launch_ypart_gate(const YGateArgs& a, hipStream_t st);

// The dense gated recurrence. One pass (see dense.hip): rows xi, kap [NS][T][DK]
// and omg [NS][T][DV], the state X [DK][DV] per stream.
struct DenseArgs {
    const void* xi; const void* kap; const void* omg;
    const float* a;          // [NS][T] gates
    const float* beta;       // [NS][T]: factor of the added product, or backwards of the output
    float* out;              // [NS][T][DV]
    const float* X0;         // [nseg][NS][..]: starting states; nullptr: zeros
    float* Xend;             // optional, the same: the states at the segments' ends
    float* segdec;           // first pass: [nseg][NS] product of the segment's gates
    const void* with;        // [NS][T][DV]: rows multiplied with the output (before beta)
    float* dot;              // [nslab][NS][T]: those products, per column slab, and
    float* inter;            // [nslab][NS][nchunk]: the part (after beta) of the chunk's starting state, summed
    int64_t NS, T, L;        // L: tokens per segment
    int64_t nchunk;          // chunks of a stream; set by the launcher
    int nseg, nslab, DK, DV;
};
struct CarryArgs {
    float* ws;               // [nseg][NS][per]: own sums in, starting states out
    const float* segdec;     // [nseg][NS]
    const float* X0;         // [NS][per] or nullptr (zeros)
    float* Xend;             // [NS][per] or nullptr
    const float* gate;       // backwards: [NS][T], the first of which decays Xend
    int64_t NS, T, per;
    int nseg;
    bool rev;
};
struct DenseGatesArgs {
    const float* G; const float* S;   // [nseg][NS][per]: states from behind, states at the starts
    const float* ST;                  // [NS][per]: after the last token
    const float* qdq; const float* kdk;  // [nslab][NS][T]
    const float* inter_q; const float* inter_k;  // [nslab][NS][nchunk]
    const float* alpha; const float* beta;
    float* dlog_alpha; float* dbeta;
    int64_t NS, T, L, per, nchunk;
    int nseg, nslab;
    bool has_dS;
};
// Tokens per chunk of the dense recurrence.
constexpr int DENSE_CHUNK = 32;
// Its passes, by what they give (S's and G's segments, and all the gradients, in one
// launch), over bf16 rows (dy's are fp32) or fp32 ones
hipError_t launch_dense_y(const DenseArgs& a, hipStream_t st);
hipError_t launch_dense_y_f32(const DenseArgs& a, hipStream_t st);
hipError_t launch_dense_s(const DenseArgs& a, hipStream_t st);
hipError_t launch_dense_s_f32(const DenseArgs& a, hipStream_t st);
hipError_t launch_dense_sg(const DenseArgs& s, const DenseArgs& g, hipStream_t st);
hipError_t launch_dense_sg_f32(const DenseArgs& s, const DenseArgs& g, hipStream_t st);
hipError_t launch_dense_grads(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st);
hipError_t launch_dense_grads_f32(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st);
struct DenseFwdArgs {
    const void* q; const void* k; const void* v; bool bf16;
    const float* alpha; const float* beta;
    const float* S0; float* S; float* y;
    int64_t NS, T;
    int dk, dv;
    void* workspace;
};
struct DenseBwdArgs {
    const void* q; const void* k; const void* v; bool bf16;
    const float* alpha; const float* beta; const float* dy;
    const float* S0; const float* dS;
    float* dq; float* dk_out; float* dv_out; float* dlog_alpha; float* dbeta; float* dS0;
    int64_t NS, T;
    int dk, dv;
    void* workspace;
};
int64_t dense_workspace_bytes(int64_t NS, int64_t T, int dk, int dv);
int64_t dense_backward_workspace_bytes(int64_t NS, int64_t T, int dk, int dv);
hipError_t launch_dense_forward(const DenseFwdArgs& a, hipStream_t st);
hipError_t launch_dense_backward(const DenseBwdArgs& a, hipStream_t st);
// X = X0 (zeros for nullptr): a call of no tokens
hipError_t launch_dense_pass_on(const float* X0, float* X, int64_t NS, int64_t per, hipStream_t st);

enum NormType { NORM_F32 = 0, NORM_BF16 = 1, NORM_E4M3 = 2 };
struct NormArgs {
    const void* x; const void* res; void* h;  // res and h: both or neither
    const float* gamma;
    void* y; float* scale;
    int64_t rows;
    int d, group, y_type;
    float eps;
    bool x_bf16, h_bf16;
    const float* bias = nullptr;
    bool mean = false;       // layer norm: the mean taken off, the bias added
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);
struct NormBwdArgs {
    const void* dy; const void* h; const void* dh; const float* gamma;
    void* dx; float* dgamma;
    float* part;             // [blocks][d]; layer norm: [blocks][2][d]
    int64_t rows;
    int d, blocks;
    float eps;
    bool g_bf16, h_bf16;     // dy, dh, dx; h
    float* dbias = nullptr;
    bool mean = false;
};
int64_t norm_bwd_blocks(int64_t rows, int d, bool mean);
hipError_t launch_norm_backward(NormBwdArgs a, hipStream_t st);

// The causal convolution: x [B,H,T,d] by strides, everything else contiguous.
struct ConvArgs {
    const void* x; const float* w; const float* bias; const void* S0; void* S;
    const uint8_t* start; const int32_t* lengths;
    void* y;
    int64_t x_b, x_h, x_t;   // elements between sequences, heads, tokens
    int64_t B, H, T;
    int d, K;
    int align;               // elements: a power of two that divides d, the strides and the tensors' addresses
    bool bf16, silu;
    // set by the launcher
    int64_t ntile;
    int tile, nvec, groups;  // groups: of 64 threads, over the pieces of all heads
};
hipError_t launch_conv(ConvArgs a, hipStream_t st);
struct ConvBwdArgs {
    const void* dy; const void* x; const float* w; const float* bias; const void* S0; const void* dS;
    const uint8_t* start; const int32_t* lengths;
    void* dx; float* dw; float* dbias; void* dS0;
    float* part;             // [B * ntile][K + 1][H * d]
    int64_t x_b, x_h, x_t, dx_b, dx_h, dx_t;
    int64_t B, H, T;
    int d, K;
    int align;
    bool bf16, silu;
    int64_t ntile;
    int tile, nvec, groups;
};
constexpr int CONV_TILE_MIN = 8;  // tokens a thread at least, of more than that: bounds the launches' wavefronts
int64_t conv_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t d, int K);
hipError_t launch_conv_backward(ConvBwdArgs a, hipStream_t st);

// The selective state-space scan: x, dt, z [B,T,D], Bm, Cm [B,T,G,N] and dy by strides, everything else
// contiguous. A tile is 64 channels of a group in one sequence (by 16 states: a wavefront's).
inline int sel_ctiles(int G, int D) { return (D / G + 63) / 64; }
inline int sel_ntiles(int N) { return (N + 15) / 16; }
inline int64_t sel_tiles(int64_t B, int G, int D) { return B * G * sel_ctiles(G, D); }
struct SelArgs {
    const void* x; const void* dt; const void* z; const void* Bm; const void* Cm;
    const float* A; const float* Dskip; const float* bias;
    const float* S0; float* S;
    const uint8_t* start; const int32_t* lengths;
    void* y;
    int64_t x_b, x_t, dt_b, dt_t, z_b, z_t, B_b, B_t, B_g, C_b, C_t, C_g;
    int64_t B, T;
    int D, G, N;
    bool bf16, softplus;
    void* workspace;
    // set by the launcher
    float* ends;             // [nseg][tiles][ntiles][1024]: what a segment adds, then where it starts
    float* steps;            // [nseg][tiles][64]: its sum of steps
    int64_t L, tiles;        // tokens per segment
    int nseg, ctiles, ntiles;
};
int64_t selective_workspace_bytes(int64_t B, int64_t T, int G, int D, int N);
hipError_t launch_selective(SelArgs a, hipStream_t st);
struct SelBwdArgs {
    const void* dy; const void* x; const void* dt; const void* z; const void* Bm; const void* Cm;
    const float* A; const float* Dskip; const float* bias;
    const float* S0; const float* dS;
    const uint8_t* start; const int32_t* lengths;
    void* dx; void* ddt; void* dz;
    float* dA; float* dB; float* dC; float* dD; float* dbias; float* dS0;
    int64_t x_b, x_t, dt_b, dt_t, z_b, z_t, B_b, B_t, B_g, C_b, C_t, C_g, dy_b, dy_t;
    int64_t B, T;
    int D, G, N;
    bool bf16, softplus;
    void* workspace;
    // set by the launcher; with the forward's ends and steps
    float* ends; float* gends; float* steps;  // gends: what a segment passes back, then what arrives at its end
    float* marks; float* msteps;  // [chunk][tiles][ntiles][1024], [chunk][tiles][64]: the segment's own state and sum of
                                  // steps in front of every chunk
    float* part_bc;          // [ctiles][B][G][T][ntiles][2][16]
    float* part_A;           // [nseg][tiles][ntiles][1024]
    float* part_D;           // [nseg][ntiles][tiles][2][64]
    int64_t L, tiles;
    int nseg, ctiles, ntiles;
};
int64_t selective_backward_workspace_bytes(int64_t B, int64_t T, int G, int D, int N);
hipError_t launch_selective_backward(SelBwdArgs a, hipStream_t st);
struct SelCarryArgs {
    float* ends; const float* steps; const float* A;
    const float* from;       // [B][D][N] or nullptr (zeros)
    int64_t tiles;
    int nseg, ntiles, ctiles, G, D, N;
    bool rev;
};

struct BalanceArgs {
    const int32_t* idx; const float* wt;  // [B,H,T,K]
    const uint8_t* mask;                  // [B,T] or nullptr
    int32_t* counts; float* mass;         // [H,N]
    int32_t* tokens;                      // [1]
    float* loss;                          // [H]
    int64_t B, H, T, K, N;
    void* workspace;
    // set by the launcher
    int64_t* fixed; int32_t* part_counts;  // [nshare][H][N]
    int32_t* bad;                          // [nshare][H]
    int32_t* kept;                         // [nshare]
    double* part;                          // [H][nblk]
    int64_t nshare, share;                 // shares of the tokens, and tokens a share
    int nrange, range, nblk, shift;        // slot ranges, and slots a range
};
int64_t balance_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t K, int64_t N);
hipError_t launch_balance(BalanceArgs a, hipStream_t st);
struct BalanceBwdArgs {
    const int32_t* idx; const uint8_t* mask; const int32_t* counts; const int32_t* tokens; const float* dloss;
    float* dwt;
    int64_t B, H, T, K, N;
    int64_t piece;           // tokens a workgroup; set by the launcher
};
constexpr int64_t BALANCE_PIECE = 4096;  // selections a workgroup of the backward's gathering form
hipError_t launch_balance_backward(BalanceBwdArgs a, hipStream_t st);

}  // namespace sdm
