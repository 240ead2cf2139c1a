// sdm_api.hip -- the C ABI (include/sdm.h): host-side validation and dispatch.
// Every check runs before any HIP call; a failing call writes nothing,
// launches nothing and records a thread-local message.
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <mutex>

#include "sdm.h"
#include "sdm_internal.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
    return code;
}

int ok() {
    g_err[0] = '\0';
    return SDM_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

int hip_fail(hipError_t e, const char* what) {
    return fail(SDM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int check_address_sizes(int q_dtype, int k_dtype, int64_t B, int64_t H, int64_t T, int64_t n_sub,
                        int64_t dh) {
    if (q_dtype != SDM_F32 && q_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown q dtype %d", q_dtype);
    if (k_dtype != q_dtype) return fail(SDM_ERR_DTYPE, "subkey dtype %d differs from q dtype %d", k_dtype, q_dtype);
    if (B < 0 || H < 0 || T < 0) return fail(SDM_ERR_SHAPE, "negative B/H/T (%lld, %lld, %lld)",
                                             (long long)B, (long long)H, (long long)T);
    if (n_sub < 1 || dh < 1) return fail(SDM_ERR_SHAPE, "n_sub and dh must be >= 1");
    if (n_sub % 16 != 0 || n_sub > 512)
        return fail(SDM_ERR_UNSUPPORTED, "n_sub=%lld: kernels cover multiples of 16 up to 512", (long long)n_sub);
    const int64_t step = q_dtype == SDM_BF16 ? 32 : 8;
    if (dh % step != 0 || dh > 256)
        return fail(SDM_ERR_UNSUPPORTED, "dh=%lld: kernels cover multiples of %lld up to 256", (long long)dh,
                    (long long)step);
    const int64_t ntile = (B * T + 15) / 16;
    if (ntile * H > 0x7FFFFFFFll) return fail(SDM_ERR_UNSUPPORTED, "too many token tiles for one launch");
    // token numbers b * T + t are kept in 32 bits on the GPU
    if (B * T > 0xFFFFFFFFll) return fail(SDM_ERR_UNSUPPORTED, "B*T=%lld: at most 2^32 - 1 tokens per call",
                                          (long long)(B * T));
    return SDM_OK;
}

}  // namespace

extern "C" {

int sdm_abi_version(void) { return SDM_ABI_VERSION; }

const char* sdm_status_string(int s) {
    switch (s) {
        case SDM_OK: return "ok";
        case SDM_ERR_NULL: return "null pointer";
        case SDM_ERR_SHAPE: return "invalid shape";
        case SDM_ERR_DTYPE: return "invalid dtype or form";
        case SDM_ERR_ALIGN: return "pointer not 16-byte aligned";
        case SDM_ERR_UNSUPPORTED: return "unsupported size";
        case SDM_ERR_HIP: return "HIP error";
        case SDM_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

const char* sdm_last_error(void) { return g_err; }

static int address_impl(const char* fn, bool idw, const void* q_w, const void* q_r, int q_dtype,
                        const void* subkeys_w, const void* subkeys_r, int k_dtype, int64_t B, int64_t H, int64_t T,
                        int64_t n_sub, int64_t dh, int64_t W, int64_t R, int32_t* idx_w, float* wt_w,
                        int32_t* idx_r, float* wt_r, float* score_w, float* score_r, void* stream) {
    int rc = check_address_sizes(q_dtype, k_dtype, B, H, T, n_sub, dh);
    if (rc) return rc;
    const int64_t N = n_sub * n_sub;
    if (W < 1 || R < 1 || W > N || R > N)
        return fail(SDM_ERR_SHAPE, "W=%lld, R=%lld must lie in [1, N=%lld]", (long long)W, (long long)R,
                    (long long)N);
    if (W > 64 || R > 64) return fail(SDM_ERR_UNSUPPORTED, "W, R <= 64 on the GPU (W=%lld, R=%lld)",
                                      (long long)W, (long long)R);
    if (B == 0 || H == 0 || T == 0) return ok();  // empty tensors may have NULL data
    if (!q_w || !q_r || !subkeys_w || !subkeys_r || !idx_w || !wt_w || !idx_r || !wt_r)
        return fail(SDM_ERR_NULL, "%s: a required pointer is NULL", fn);
    const void* ptrs[] = {q_w, q_r, subkeys_w, subkeys_r, idx_w, wt_w, idx_r, wt_r};
    for (const void* p : ptrs)
        if (!aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    if ((score_w && !aligned16(score_w)) || (score_r && !aligned16(score_r)))
        return fail(SDM_ERR_ALIGN, "%s: score pointer not 16-byte aligned", fn);
    sdm::AddressArgs a{};
    a.q[0] = q_w; a.q[1] = q_r;
    a.K[0] = subkeys_w; a.K[1] = subkeys_r;
    a.idx[0] = idx_w; a.idx[1] = idx_r;
    a.wt[0] = wt_w; a.wt[1] = wt_r;
    a.score[0] = score_w; a.score[1] = score_r;
    a.k[0] = (int)W; a.k[1] = (int)R;
    a.half_out = nullptr;
    a.B = B; a.H = H; a.T = T; a.n = (int)n_sub; a.dh = (int)dh;
    a.nbranch = 2;
    a.bf16 = q_dtype == SDM_BF16;
    a.idw = idw;
    hipError_t e = sdm::launch_address(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

static int half_scores_impl(const char* fn, bool idw, const void* q, int q_dtype, const void* subkeys, int k_dtype,
                            int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh, float* half, void* stream) {
    int rc = check_address_sizes(q_dtype, k_dtype, B, H, T, n_sub, dh);
    if (rc) return rc;
    if (B == 0 || H == 0 || T == 0) return ok();
    if (!q || !subkeys || !half) return fail(SDM_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned16(q) || !aligned16(subkeys) || !aligned16(half))
        return fail(SDM_ERR_ALIGN, "%s: pointer not 16-byte aligned", fn);
    sdm::AddressArgs a{};
    a.q[0] = q; a.K[0] = subkeys;
    a.k[0] = 1;
    a.half_out = half;
    a.B = B; a.H = H; a.T = T; a.n = (int)n_sub; a.dh = (int)dh;
    a.nbranch = 1;
    a.bf16 = q_dtype == SDM_BF16;
    a.idw = idw;
    hipError_t e = sdm::launch_address(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

int sdm_address(const void* q_w, const void* q_r, int q_dtype, const void* subkeys_w, const void* subkeys_r,
                int k_dtype, int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh, int64_t W, int64_t R,
                int32_t* idx_w, float* wt_w, int32_t* idx_r, float* wt_r, float* score_w, float* score_r,
                void* stream) {
    return address_impl("sdm_address", false, q_w, q_r, q_dtype, subkeys_w, subkeys_r, k_dtype, B, H, T, n_sub, dh,
                        W, R, idx_w, wt_w, idx_r, wt_r, score_w, score_r, stream);
}

int sdm_address_idw(const void* q_w, const void* q_r, int q_dtype, const void* subkeys_w, const void* subkeys_r,
                    int k_dtype, int64_t B, int64_t H, int64_t T, int64_t n_sub, int64_t dh, int64_t W, int64_t R,
                    int32_t* idx_w, float* wt_w, int32_t* idx_r, float* wt_r, float* score_w, float* score_r,
                    void* stream) {
    return address_impl("sdm_address_idw", true, q_w, q_r, q_dtype, subkeys_w, subkeys_r, k_dtype, B, H, T, n_sub,
                        dh, W, R, idx_w, wt_w, idx_r, wt_r, score_w, score_r, stream);
}

int sdm_debug_half_scores(const void* q, int q_dtype, const void* subkeys, int k_dtype, int64_t B, int64_t H,
                          int64_t T, int64_t n_sub, int64_t dh, float* half, void* stream) {
    return half_scores_impl("sdm_debug_half_scores", false, q, q_dtype, subkeys, k_dtype, B, H, T, n_sub, dh, half,
                            stream);
}

int sdm_debug_half_scores_idw(const void* q, int q_dtype, const void* subkeys, int k_dtype, int64_t B, int64_t H,
                              int64_t T, int64_t n_sub, int64_t dh, float* half, void* stream) {
    return half_scores_impl("sdm_debug_half_scores_idw", true, q, q_dtype, subkeys, k_dtype, B, H, T, n_sub, dh,
                            half, stream);
}

int sdm_state_init(const float* M0, void* M, int m_dtype, int64_t B, int64_t H, int64_t N, int64_t dv,
                   void* stream) {
    if (m_dtype != SDM_F32 && m_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown table dtype %d", m_dtype);
    if (B < 0 || H < 0 || N < 1 || dv < 1) return fail(SDM_ERR_SHAPE, "sdm_state_init: invalid sizes");
    if (dv % 4 != 0) return fail(SDM_ERR_UNSUPPORTED, "sdm_state_init: dv must be a multiple of 4");
    if (B == 0 || H == 0) return ok();
    if (!M0 || !M) return fail(SDM_ERR_NULL, "sdm_state_init: NULL pointer");
    if (!aligned16(M0) || !aligned16(M)) return fail(SDM_ERR_ALIGN, "sdm_state_init: pointer not 16-byte aligned");
    hipError_t e = sdm::launch_state_init(M0, M, m_dtype == SDM_BF16, B, H * N * dv,
                                          static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "sdm_state_init launch");
    return ok();
}

int64_t sdm_scan_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R, int64_t dv) {
    if (B < 0 || H < 0 || T < 0 || W < 1 || R < 1 || W > 256 || R > 256 || dv < 4 || dv % 4) return -1;
    if (B == 0 || H == 0 || T == 0) return 0;
    return sdm::scan_workspace_bytes(B * H, T, (int)W, (int)R, (int)dv);
}

}  // extern "C"

namespace {

// Shared checks of the scan entry points (sizes, dtypes, pointers, alignment,
// workspace). 0 when the call may launch; NO_WORK when there is no work (the
// call succeeds and launches nothing); otherwise the status code.
constexpr int NO_WORK = -1;
int check_scan(const char* fn, const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r,
               const float* wt_r, int64_t R, const float* alpha, const float* beta, const void* v, int v_dtype,
               int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv, int form, int m_dtype = SDM_F32) {
    if (v_dtype != SDM_F32 && v_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown v dtype %d", v_dtype);
    if (m_dtype != SDM_F32 && m_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown table dtype %d", m_dtype);
    if (form != SDM_DELTA_EQ4 && form != SDM_DELTA_FIG2) return fail(SDM_ERR_DTYPE, "unknown delta form %d", form);
    if (B < 0 || H < 0 || T < 0 || N < 1 || dv < 1) return fail(SDM_ERR_SHAPE, "%s: invalid sizes", fn);
    if (W < 1 || R < 1 || W > N || R > N)
        return fail(SDM_ERR_SHAPE, "W=%lld, R=%lld must lie in [1, N=%lld]", (long long)W, (long long)R,
                    (long long)N);
    if (W > 256 || R > 256) return fail(SDM_ERR_UNSUPPORTED, "W, R <= 256 on the GPU");
    if (N > (1 << 18)) return fail(SDM_ERR_UNSUPPORTED, "N=%lld: at most 2^18 slots", (long long)N);
    if (dv % 4 != 0) return fail(SDM_ERR_UNSUPPORTED, "dv=%lld must be a multiple of 4", (long long)dv);
    if (m_dtype == SDM_BF16 && dv % 8 != 0)
        return fail(SDM_ERR_UNSUPPORTED, "dv=%lld must be a multiple of 8 for a bf16 table", (long long)dv);
    if (N * dv * 4 >= (1ll << 31))
        return fail(SDM_ERR_UNSUPPORTED, "one stream's table (N*dv*4 = %lld bytes) must stay below 2 GiB",
                    (long long)(N * dv * 4));
    if (!sdm::scan_geometry(B * H > 0 ? B * H : 1, (int)W, (int)R, (int)dv, m_dtype == SDM_BF16, nullptr,
                            nullptr))
        return fail(SDM_ERR_UNSUPPORTED, "no scan kernel covers W=%lld, R=%lld, dv=%lld", (long long)W,
                    (long long)R, (long long)dv);
    if ((B * H + 7) / 8 * 8 * (dv / 4) > 0x7FFFFFFFll)
        return fail(SDM_ERR_UNSUPPORTED, "too many streams for one launch");
    if (B == 0 || H == 0 || T == 0) return NO_WORK;  // empty tensors may have NULL data
    if (!idx_w || !wt_w || !idx_r || !wt_r || !alpha || !beta || !v)
        return fail(SDM_ERR_NULL, "%s: a required pointer is NULL", fn);
    const void* ptrs[] = {idx_w, wt_w, idx_r, wt_r, alpha, beta, v};
    for (const void* p : ptrs)
        if (!aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    return 0;
}

int check_buffers(const char* fn, std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs) {
        if (!p) return fail(SDM_ERR_NULL, "%s: a required pointer is NULL", fn);
        if (!aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    }
    return 0;
}

int check_workspace(void* workspace, int64_t workspace_bytes, int64_t need) {
    if (!workspace || workspace_bytes < need)
        return fail(SDM_ERR_WORKSPACE, "workspace of %lld bytes needed, %lld given", (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    if (!aligned16(workspace)) return fail(SDM_ERR_ALIGN, "workspace not 16-byte aligned");
    return 0;
}

int scan_forward_impl(const char* fn, const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r,
                      const float* wt_r, int64_t R, const float* alpha, const float* beta, const void* v,
                      int v_dtype, void* M, int m_dtype, float* y, float* snap, bool save, int64_t B, int64_t H,
                      int64_t T, int64_t N, int64_t dv, int form, void* workspace, int64_t workspace_bytes,
                      void* stream) {
    int rc = check_scan(fn, idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, B, H, T, N, dv, form,
                        m_dtype);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if ((rc = check_buffers(fn, {M, y}))) return rc;
    if (save && (rc = check_buffers(fn, {snap}))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes,
                              sdm::scan_workspace_bytes(B * H, T, (int)W, (int)R, (int)dv))))
        return rc;
    sdm::ScanArgs a{};
    a.idx_w = idx_w; a.wt_w = wt_w; a.W = (int)W;
    a.idx_r = idx_r; a.wt_r = wt_r; a.R = (int)R;
    a.alpha = alpha; a.beta = beta;
    a.v = v; a.v_bf16 = v_dtype == SDM_BF16;
    a.M = M; a.m_bf16 = m_dtype == SDM_BF16; a.y = y;
    a.NS = B * H; a.T = T; a.N = N; a.dv = (int)dv;
    a.form = form;
    a.workspace = workspace;
    a.snap = save ? snap : nullptr;
    hipError_t e = sdm::launch_scan(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

}  // namespace

extern "C" {

int sdm_scan_forward(const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r, const float* wt_r,
                     int64_t R, const float* alpha, const float* beta, const void* v, int v_dtype, void* M,
                     int m_dtype, float* y, int64_t B, int64_t H, int64_t T, int64_t N, int64_t dv, int form,
                     void* workspace, int64_t workspace_bytes, void* stream) {
    return scan_forward_impl("sdm_scan_forward", idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, M,
                             m_dtype, y, nullptr, false, B, H, T, N, dv, form, workspace, workspace_bytes, stream);
}

int64_t sdm_scan_gated_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R, int64_t dv) {
    const int64_t b = sdm_scan_workspace_bytes(B, H, T, W, R, dv);
    if (b <= 0) return b;
    return (b + 255) / 256 * 256 + B * H * T * dv * 4;  // + y, where the call keeps it itself
}

int sdm_scan_forward_gated(const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r,
                           const float* wt_r, int64_t R, const float* alpha, const float* beta, const void* v,
                           int v_dtype, void* M, int m_dtype, float* y, const float* gamma, const void* g,
                           int g_dtype, float eps, float* o, int64_t B, int64_t H, int64_t T, int64_t N,
                           int64_t dv, int form, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_scan_forward_gated";
    int rc = check_scan(fn, idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, B, H, T, N, dv, form,
                        m_dtype);
    if (g_dtype != SDM_F32 && g_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown gate dtype %d", g_dtype);
    if (!(eps >= 0.f)) return fail(SDM_ERR_SHAPE, "%s: eps must be >= 0", fn);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if (B * H * T > 0xFFFFFFFFll)
        return fail(SDM_ERR_UNSUPPORTED, "B*H*T=%lld: at most 2^32 - 1 rows per call", (long long)(B * H * T));
    if ((rc = check_buffers(fn, {M, gamma, g, o}))) return rc;
    if (y && !aligned16(y)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, (void*)y);
    if (o == y) return fail(SDM_ERR_SHAPE, "%s: o may not alias y", fn);
    const int64_t scan_ws = sdm::scan_workspace_bytes(B * H, T, (int)W, (int)R, (int)dv);
    if ((rc = check_workspace(workspace, workspace_bytes, (scan_ws + 255) / 256 * 256 + B * H * T * dv * 4)))
        return rc;
    sdm::GateArgs ga{};
    ga.gamma = gamma; ga.g = g; ga.o = o; ga.eps = eps; ga.H = H; ga.g_bf16 = g_dtype == SDM_BF16;
    const bool fused = sdm::scan_fuses_gate(B * H, T, (int)W, (int)R, (int)dv, m_dtype == SDM_BF16, form);
    // where the scan stores y itself and the caller passed none, y goes to the workspace's tail
    float* yy = y ? y : reinterpret_cast<float*>(static_cast<char*>(workspace) + (scan_ws + 255) / 256 * 256);
    sdm::ScanArgs a{};
    a.idx_w = idx_w; a.wt_w = wt_w; a.W = (int)W;
    a.idx_r = idx_r; a.wt_r = wt_r; a.R = (int)R;
    a.alpha = alpha; a.beta = beta;
    a.v = v; a.v_bf16 = v_dtype == SDM_BF16;
    a.M = M; a.m_bf16 = m_dtype == SDM_BF16;
    a.y = fused ? y : yy;
    a.NS = B * H; a.T = T; a.N = N; a.dv = (int)dv;
    a.form = form;
    a.workspace = workspace;
    a.gate = fused ? &ga : nullptr;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e = sdm::launch_scan(a, st);
    if (e != hipSuccess) return hip_fail(e, fn);
    if (!fused) {
        sdm::OutGateArgs og{};
        og.y = yy; og.gamma = gamma; og.g = g; og.o = o; og.eps = eps;
        og.rows = B * H * T; og.T = T; og.H = H; og.dv = (int)dv; og.g_bf16 = ga.g_bf16;
        e = sdm::launch_output_gate(og, st);
        if (e != hipSuccess) return hip_fail(e, fn);
    }
    return ok();
}

}  // extern "C"

namespace {

// The scan's scratch (plan records, partial y, counters) for callers that cannot
// allocate: one array per GPU, kept until the process ends. Host code uses its
// device address from hipGetSymbolAddress, taken once per device.
constexpr int64_t SCRATCH_BYTES = 64ll << 20;
__device__ __align__(256) unsigned char scratch[SCRATCH_BYTES];

constexpr int MAX_DEVICES = 64;
std::once_flag g_scratch_once[MAX_DEVICES];
void* g_scratch_ptr[MAX_DEVICES];
hipError_t g_scratch_err[MAX_DEVICES];

// Device address of this GPU's scratch array (nullptr and the error on failure).
void* scratch_of(int dev, hipError_t* err) {
    std::call_once(g_scratch_once[dev], [dev] {
        int cur = 0;
        hipError_t e = hipGetDevice(&cur);
        if (e == hipSuccess && cur != dev) e = hipSetDevice(dev);
        void* p = nullptr;
        if (e == hipSuccess) e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (cur != dev) (void)hipSetDevice(cur);
        g_scratch_err[dev] = e;
        g_scratch_ptr[dev] = e == hipSuccess ? p : nullptr;
    });
    *err = g_scratch_err[dev];
    return g_scratch_ptr[dev];
}

}  // namespace

extern "C" {

int sdm_scan_forward_noalloc(const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r,
                             const float* wt_r, int64_t R, const float* alpha, const float* beta, const void* v,
                             int v_dtype, void* M, int m_dtype, float* y, int64_t B, int64_t H, int64_t T,
                             int64_t N, int64_t dv, int form, void* stream) {
    const char* fn = "sdm_scan_forward_noalloc";
    int rc = check_scan(fn, idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, B, H, T, N, dv, form,
                        m_dtype);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if ((rc = check_buffers(fn, {M, y}))) return rc;
    const int64_t tc = sdm::scan_tokens_within(B * H, T, (int)W, (int)R, (int)dv, m_dtype == SDM_BF16, form,
                                               SCRATCH_BYTES);
    if (tc < 1)
        return fail(SDM_ERR_UNSUPPORTED,
                    "%s: B*H=%lld streams need more than the %lld-byte scratch for even one token per launch",
                    fn, (long long)(B * H), (long long)SCRATCH_BYTES);
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess && stream) e = hipStreamGetDevice(static_cast<hipStream_t>(stream), &dev);
    if (e != hipSuccess) return hip_fail(e, fn);
    if (dev < 0 || dev >= MAX_DEVICES) return fail(SDM_ERR_UNSUPPORTED, "%s: device %d out of range", fn, dev);
    void* ws = scratch_of(dev, &e);
    if (!ws) return hip_fail(e, "sdm_scan_forward_noalloc (scratch address)");
    sdm::ScanArgs a{};
    a.idx_w = idx_w; a.wt_w = wt_w; a.W = (int)W;
    a.idx_r = idx_r; a.wt_r = wt_r; a.R = (int)R;
    a.alpha = alpha; a.beta = beta;
    a.v = v; a.v_bf16 = v_dtype == SDM_BF16;
    a.M = M; a.m_bf16 = m_dtype == SDM_BF16; a.y = y;
    a.NS = B * H; a.T = T; a.N = N; a.dv = (int)dv;
    a.form = form;
    a.workspace = ws;
    a.snap = nullptr;
    a.max_tokens = tc;
    e = sdm::launch_scan(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

int64_t sdm_scan_snapshot_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t dv) {
    if (B < 0 || H < 0 || T < 0 || W < 1 || dv < 1) return -1;
    return B * H * T * W * dv * 4;
}

int sdm_scan_forward_save(const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r,
                          const float* wt_r, int64_t R, const float* alpha, const float* beta, const void* v,
                          int v_dtype, float* M, float* y, float* snap, int64_t B, int64_t H, int64_t T, int64_t N,
                          int64_t dv, int form, void* workspace, int64_t workspace_bytes, void* stream) {
    return scan_forward_impl("sdm_scan_forward_save", idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, M,
                             SDM_F32, y, snap, true, B, H, T, N, dv, form, workspace, workspace_bytes, stream);
}

int64_t sdm_scan_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t W, int64_t R, int64_t dv) {
    if (B < 0 || H < 0 || T < 0 || W < 1 || R < 1 || W > 256 || R > 256 || dv < 4 || dv % 4) return -1;
    if (B == 0 || H == 0 || T == 0) return 0;
    return sdm::scan_backward_workspace_bytes(B * H, T, (int)W, (int)R, (int)dv);
}

int sdm_scan_backward(const int32_t* idx_w, const float* wt_w, int64_t W, const int32_t* idx_r, const float* wt_r,
                      int64_t R, const float* alpha, const float* beta, const void* v, int v_dtype,
                      const float* snap, const float* dy, float* M, float* dM, float* dv_out, float* dalpha,
                      float* dbeta, float* dwt_w, float* dwt_r, int64_t B, int64_t H, int64_t T, int64_t N,
                      int64_t dv, int form, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_scan_backward";
    int rc = check_scan(fn, idx_w, wt_w, W, idx_r, wt_r, R, alpha, beta, v, v_dtype, B, H, T, N, dv, form);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if (!sdm::scan_backward_geometry(B * H, (int)W, (int)R, (int)dv))
        return fail(SDM_ERR_UNSUPPORTED, "no backward kernel covers W=%lld, R=%lld, dv=%lld", (long long)W,
                    (long long)R, (long long)dv);
    if ((rc = check_buffers(fn, {snap, dy, M, dM, dv_out, dalpha, dbeta, dwt_w, dwt_r}))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes,
                              sdm::scan_backward_workspace_bytes(B * H, T, (int)W, (int)R, (int)dv))))
        return rc;
    sdm::BwdArgs a{};
    a.idx_w = idx_w; a.wt_w = wt_w; a.W = (int)W;
    a.idx_r = idx_r; a.wt_r = wt_r; a.R = (int)R;
    a.alpha = alpha; a.beta = beta;
    a.v = v; a.v_bf16 = v_dtype == SDM_BF16;
    a.snap = snap; a.dy = dy; a.M = M; a.dM = dM;
    a.dv_out = dv_out; a.dalpha = dalpha; a.dbeta = dbeta; a.dwt_w = dwt_w; a.dwt_r = dwt_r;
    a.NS = B * H; a.T = T; a.N = N; a.dv = (int)dv;
    a.form = form;
    a.workspace = workspace;
    hipError_t e = sdm::launch_scan_backward(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

int sdm_gates(const void* x, int x_dtype, const void* W_a, const void* W_b, int w_dtype, const float* b_dt,
              const float* A, int64_t B, int64_t T, int64_t d, int64_t H, float* alpha, float* beta, void* stream) {
    const char* fn = "sdm_gates";
    if (x_dtype != SDM_F32 && x_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown x dtype %d", x_dtype);
    if (w_dtype != x_dtype) return fail(SDM_ERR_DTYPE, "weight dtype %d differs from x dtype %d", w_dtype, x_dtype);
    if (B < 0 || T < 0 || d < 1 || H < 1) return fail(SDM_ERR_SHAPE, "%s: invalid sizes", fn);
    const int64_t step = x_dtype == SDM_BF16 ? 32 : 8;
    if (d % step != 0 || d > (1 << 20))
        return fail(SDM_ERR_UNSUPPORTED, "d=%lld: a multiple of %lld up to 2^20", (long long)d, (long long)step);
    if (H > 4096) return fail(SDM_ERR_UNSUPPORTED, "H=%lld: at most 4096 heads", (long long)H);
    if (B * T > 0xFFFFFFFFll) return fail(SDM_ERR_UNSUPPORTED, "B*T=%lld: at most 2^32 - 1 tokens per call",
                                          (long long)(B * T));
    if (B == 0 || T == 0) return ok();
    int rc = check_buffers(fn, {x, W_a, W_b, b_dt, A, alpha, beta});
    if (rc) return rc;
    sdm::GatesArgs a{};
    a.x = x; a.Wa = W_a; a.Wb = W_b; a.bdt = b_dt; a.A = A; a.alpha = alpha; a.beta = beta;
    a.B = B; a.T = T; a.d = (int)d; a.H = (int)H; a.bf16 = x_dtype == SDM_BF16;
    hipError_t e = sdm::launch_gates(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

int sdm_output_gate(const float* y, const float* gamma, const void* g, int g_dtype, float eps, int64_t B,
                    int64_t H, int64_t T, int64_t dv, float* o, void* stream) {
    const char* fn = "sdm_output_gate";
    if (g_dtype != SDM_F32 && g_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "unknown gate dtype %d", g_dtype);
    if (B < 0 || H < 1 || T < 0 || dv < 1 || !(eps >= 0.f)) return fail(SDM_ERR_SHAPE, "%s: invalid sizes or eps", fn);
    if (dv % 4 != 0) return fail(SDM_ERR_UNSUPPORTED, "dv=%lld must be a multiple of 4", (long long)dv);
    if (B * H * T > 0xFFFFFFFFll)
        return fail(SDM_ERR_UNSUPPORTED, "B*H*T=%lld: at most 2^32 - 1 rows per call", (long long)(B * H * T));
    if (B == 0 || T == 0) return ok();
    int rc = check_buffers(fn, {y, gamma, g, o});
    if (rc) return rc;
    sdm::OutGateArgs a{};
    a.y = y; a.gamma = gamma; a.g = g; a.o = o; a.eps = eps;
    a.rows = B * H * T; a.T = T; a.H = H; a.dv = (int)dv; a.g_bf16 = g_dtype == SDM_BF16;
    hipError_t e = sdm::launch_output_gate(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, fn);
    return ok();
}

int sdm_state_init_backward(const float* dM, float* dM0, int64_t B, int64_t H, int64_t N, int64_t dv,
                            void* stream) {
    if (B < 0 || H < 0 || N < 1 || dv < 1) return fail(SDM_ERR_SHAPE, "sdm_state_init_backward: invalid sizes");
    if (dv % 4 != 0) return fail(SDM_ERR_UNSUPPORTED, "sdm_state_init_backward: dv must be a multiple of 4");
    if (H == 0) return ok();
    if (B == 0) return fail(SDM_ERR_SHAPE, "sdm_state_init_backward: B must be >= 1");
    int rc = check_buffers("sdm_state_init_backward", {dM, dM0});
    if (rc) return rc;
    hipError_t e = sdm::launch_state_init_backward(dM, dM0, B, H * N * dv, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "sdm_state_init_backward launch");
    return ok();
}

}  // extern "C"

namespace {

// Sizes, dtype and the row tensors of the dense recurrence (0, NO_WORK for no
// streams, or the status).
int check_dense(const char* fn, int in_dtype, int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv) {
    if (in_dtype != SDM_F32 && in_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown dtype %d", fn, in_dtype);
    if (B < 0 || H < 0 || T < 0 || dk < 1 || dv < 1) return fail(SDM_ERR_SHAPE, "%s: invalid sizes", fn);
    if (dk % 8 != 0 || dv % 8 != 0 || dk > 256 || dv > 256)
        return fail(SDM_ERR_UNSUPPORTED, "%s: dk=%lld, dv=%lld: multiples of 8 up to 256", fn, (long long)dk,
                    (long long)dv);
    // B, H and T below 2^31 each, so that the products below stay in 64 bits
    if (B > 0x7FFFFFFFll || H > 0x7FFFFFFFll || T > 0x7FFFFFFFll || B * H > 0x7FFFFFFFll ||
        B * H * 8 * ((T + 63) / 64) > 0x7FFFFFFFll ||
        // fewer than 2^32 threads a launch: three passes of 512 a segment and slab; 4 elements a thread
        B * H * ((T + 511) / 512) * (((dk > dv ? dk : dv) + 63) / 64) >= 1ll << 21 ||
        B * H * dk * dv >= (1ll << 34) - 1024)
        return fail(SDM_ERR_UNSUPPORTED, "%s: too many streams or tokens for one launch", fn);
    return B == 0 || H == 0 ? NO_WORK : 0;
}

}  // namespace

extern "C" {

int64_t sdm_dense_scan_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv) {
    const int rc = check_dense("sdm_dense_scan_workspace_bytes", SDM_F32, B, H, T, dk, dv);
    if (rc == NO_WORK || (rc == 0 && T == 0)) return 0;
    if (rc) return -1;
    return sdm::dense_workspace_bytes(B * H, T, (int)dk, (int)dv);
}

int sdm_dense_scan_forward(const void* q, const void* k, const void* v, int in_dtype, const float* alpha,
                           const float* beta, const float* S0, float* S, float* y, int64_t B, int64_t H, int64_t T,
                           int64_t dk, int64_t dv, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_dense_scan_forward";
    int rc = check_dense(fn, in_dtype, B, H, T, dk, dv);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if (T > 0 && (rc = check_buffers(fn, {q, k, v, alpha, beta, y}))) return rc;
    if (S0 && !aligned16(S0)) return fail(SDM_ERR_ALIGN, "%s: S0 not 16-byte aligned", fn);
    if (S && !aligned16(S)) return fail(SDM_ERR_ALIGN, "%s: S not 16-byte aligned", fn);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (T == 0) {
        if (!S || S == S0) return ok();
        e = sdm::launch_dense_pass_on(S0, S, B * H, dk * dv, st);
        return e == hipSuccess ? ok() : hip_fail(e, fn);
    }
    const int64_t need = sdm::dense_workspace_bytes(B * H, T, (int)dk, (int)dv);
    if (need > 0 && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
    sdm::DenseFwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.bf16 = in_dtype == SDM_BF16;
    a.alpha = alpha; a.beta = beta; a.S0 = S0; a.S = S; a.y = y;
    a.NS = B * H; a.T = T; a.dk = (int)dk; a.dv = (int)dv;
    a.workspace = workspace;
    e = sdm::launch_dense_forward(a, st);
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

int64_t sdm_dense_scan_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t dk, int64_t dv) {
    const int rc = check_dense("sdm_dense_scan_backward_workspace_bytes", SDM_F32, B, H, T, dk, dv);
    if (rc == NO_WORK || (rc == 0 && T == 0)) return 0;
    if (rc) return -1;
    return sdm::dense_backward_workspace_bytes(B * H, T, (int)dk, (int)dv);
}

int sdm_dense_scan_backward(const void* q, const void* k, const void* v, int in_dtype, const float* alpha,
                            const float* beta, const float* dy, const float* S0, const float* dS, float* dq,
                            float* dk_out, float* dv_out, float* dlog_alpha, float* dbeta, float* dS0, int64_t B,
                            int64_t H, int64_t T, int64_t dk, int64_t dv, void* workspace, int64_t workspace_bytes,
                            void* stream) {
    const char* fn = "sdm_dense_scan_backward";
    int rc = check_dense(fn, in_dtype, B, H, T, dk, dv);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    if (T > 0 && (rc = check_buffers(fn, {q, k, v, alpha, beta, dy, dq, dk_out, dv_out, dlog_alpha, dbeta}))) return rc;
    const void* opt[] = {S0, dS, dS0};
    for (const void* p : opt)
        if (p && !aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    if (T == 0) {
        if (!dS0 || dS0 == dS) return ok();
        e = sdm::launch_dense_pass_on(dS, dS0, B * H, dk * dv, st);
        return e == hipSuccess ? ok() : hip_fail(e, fn);
    }
    if ((rc = check_workspace(workspace, workspace_bytes,
                              sdm::dense_backward_workspace_bytes(B * H, T, (int)dk, (int)dv))))
        return rc;
    sdm::DenseBwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.bf16 = in_dtype == SDM_BF16;
    a.alpha = alpha; a.beta = beta; a.dy = dy; a.S0 = S0; a.dS = dS;
    a.dq = dq; a.dk_out = dk_out; a.dv_out = dv_out; a.dlog_alpha = dlog_alpha; a.dbeta = dbeta; a.dS0 = dS0;
    a.NS = B * H; a.T = T; a.dk = (int)dk; a.dv = (int)dv;
    a.workspace = workspace;
    e = sdm::launch_dense_backward(a, st);
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

}  // extern "C"

namespace {

int check_norm_sizes(const char* fn, int64_t rows, int64_t d, float eps) {
    if (rows < 0 || d < 1 || !(eps >= 0.f)) return fail(SDM_ERR_SHAPE, "%s: invalid sizes or eps", fn);
    if (d > 16384) return fail(SDM_ERR_UNSUPPORTED, "%s: d=%lld: at most 16384", fn, (long long)d);
    if (rows > 0x7FFFFFFFll) return fail(SDM_ERR_UNSUPPORTED, "%s: at most 2^31 - 1 rows per call", fn);
    return 0;
}

}  // namespace

namespace {

// Outputs (NULL: not given) at addresses of their own, and at none of the inputs that are read beside their stores
int check_own(const char* fn, std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
    for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
        for (const void* const* p = outs.begin(); *o && p != o; ++p)
            if (*p == *o) return fail(SDM_ERR_SHAPE, "%s: two outputs at one address", fn);
        for (const void* i : ins)
            if (*o && i == *o) return fail(SDM_ERR_SHAPE, "%s: an output may not alias an input", fn);
    }
    return 0;
}

int norm_impl(const char* fn, bool mean, const void* x, int x_dtype, const void* res, void* h, int h_dtype,
              const float* gamma, const float* bias, float eps, int64_t rows, int64_t d, void* y, int y_dtype,
              float* scale, int64_t group, void* stream) {
    if (x_dtype != SDM_F32 && x_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown x dtype %d", fn, x_dtype);
    if (h_dtype != SDM_F32 && h_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown h dtype %d", fn, h_dtype);
    if (y_dtype != SDM_F32 && y_dtype != SDM_BF16 && y_dtype != SDM_E4M3)
        return fail(SDM_ERR_DTYPE, "%s: unknown y dtype %d", fn, y_dtype);
    int rc = check_norm_sizes(fn, rows, d, eps);
    if (rc) return rc;
    if (group != 0) {
        if (y_dtype != SDM_E4M3) return fail(SDM_ERR_SHAPE, "%s: groups belong to an e4m3 output", fn);
        if (group < 32 || group > 512 || (group & (group - 1)) != 0 || d % group != 0)
            return fail(SDM_ERR_UNSUPPORTED, "%s: group=%lld: 0, or a power of two from 32 to 512 that divides d=%lld",
                        fn, (long long)group, (long long)d);
    }
    if (rows == 0) return ok();
    if ((rc = check_buffers(fn, {x, gamma, y}))) return rc;
    if ((res == nullptr) != (h == nullptr)) return fail(SDM_ERR_NULL, "%s: res and h go together", fn);
    if (res && (rc = check_buffers(fn, {res, h}))) return rc;
    if (bias && (rc = check_buffers(fn, {bias}))) return rc;
    if (y_dtype == SDM_E4M3 && (rc = check_buffers(fn, {scale}))) return rc;
    if (y == x || y == h || (res && y == res)) return fail(SDM_ERR_SHAPE, "%s: y may not alias x, res or h", fn);
    if (h && h == x && x_dtype != h_dtype) return fail(SDM_ERR_SHAPE, "%s: h may alias x only in the same dtype", fn);
    if (mean) {  // (a row's inputs and outputs go by rows, scales and parameters do not)
        const void* sc = y_dtype == SDM_E4M3 ? scale : nullptr;
        if ((rc = check_own(fn, {y, h, sc}, {gamma, bias})) || (rc = check_own(fn, {sc}, {x, res}))) return rc;
    }
    sdm::NormArgs a{};
    a.x = x; a.res = res; a.h = h; a.gamma = gamma; a.y = y; a.scale = scale;
    a.rows = rows; a.d = (int)d; a.group = (int)group; a.eps = eps;
    a.y_type = y_dtype == SDM_E4M3 ? sdm::NORM_E4M3 : y_dtype == SDM_BF16 ? sdm::NORM_BF16 : sdm::NORM_F32;
    a.x_bf16 = x_dtype == SDM_BF16; a.h_bf16 = h_dtype == SDM_BF16;
    a.bias = bias; a.mean = mean;
    hipError_t e = sdm::launch_norm(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

int64_t norm_backward_bytes(bool mean, int64_t rows, int64_t d) {
    if (rows < 0 || d < 1 || d > 16384 || rows > 0x7FFFFFFFll) return -1;
    return rows == 0 ? 0 : sdm::norm_bwd_blocks(rows, (int)d, mean) * d * (mean ? 8 : 4);
}

int norm_backward_impl(const char* fn, bool mean, const void* dy, const void* dh, int g_dtype, const void* h,
                       int h_dtype, const float* gamma, float eps, int64_t rows, int64_t d, void* dx, float* dgamma,
                       float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    if (g_dtype != SDM_F32 && g_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown gradient dtype %d", fn, g_dtype);
    if (h_dtype != SDM_F32 && h_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown h dtype %d", fn, h_dtype);
    int rc = check_norm_sizes(fn, rows, d, eps);
    if (rc) return rc;
    if (rows == 0) return ok();
    if ((rc = check_buffers(fn, {dy, h, gamma, dx, dgamma}))) return rc;
    if (dh && !aligned16(dh)) return fail(SDM_ERR_ALIGN, "%s: dh not 16-byte aligned", fn);
    if (dbias && !aligned16(dbias)) return fail(SDM_ERR_ALIGN, "%s: dbias not 16-byte aligned", fn);
    if (dx == h && g_dtype != h_dtype) return fail(SDM_ERR_SHAPE, "%s: dx may alias h only in the same dtype", fn);
    if ((rc = check_workspace(workspace, workspace_bytes, norm_backward_bytes(mean, rows, d)))) return rc;
    if (mean && ((rc = check_own(fn, {dx, dgamma, dbias}, {})) || (rc = check_own(fn, {dx}, {gamma})))) return rc;
    sdm::NormBwdArgs a{};
    a.dy = dy; a.dh = dh; a.h = h; a.gamma = gamma; a.dx = dx; a.dgamma = dgamma;
    a.part = static_cast<float*>(workspace);
    a.rows = rows; a.d = (int)d; a.eps = eps;
    a.g_bf16 = g_dtype == SDM_BF16; a.h_bf16 = h_dtype == SDM_BF16;
    a.dbias = dbias; a.mean = mean;
    hipError_t e = sdm::launch_norm_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

}  // namespace

extern "C" {

int sdm_residual_norm(const void* x, int x_dtype, const void* res, void* h, int h_dtype, const float* gamma,
                      float eps, int64_t rows, int64_t d, void* y, int y_dtype, float* scale, int64_t group,
                      void* stream) {
    return norm_impl("sdm_residual_norm", false, x, x_dtype, res, h, h_dtype, gamma, nullptr, eps, rows, d, y, y_dtype,
                     scale, group, stream);
}

int64_t sdm_residual_norm_backward_workspace_bytes(int64_t rows, int64_t d) { return norm_backward_bytes(false, rows, d); }

int sdm_residual_norm_backward(const void* dy, const void* dh, int g_dtype, const void* h, int h_dtype,
                               const float* gamma, float eps, int64_t rows, int64_t d, void* dx, float* dgamma,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    return norm_backward_impl("sdm_residual_norm_backward", false, dy, dh, g_dtype, h, h_dtype, gamma, eps, rows, d, dx,
                              dgamma, nullptr, workspace, workspace_bytes, stream);
}

int sdm_residual_layer_norm(const void* x, int x_dtype, const void* res, void* h, int h_dtype, const float* gamma,
                            const float* bias, float eps, int64_t rows, int64_t d, void* y, int y_dtype, float* scale,
                            int64_t group, void* stream) {
    return norm_impl("sdm_residual_layer_norm", true, x, x_dtype, res, h, h_dtype, gamma, bias, eps, rows, d, y, y_dtype,
                     scale, group, stream);
}

int64_t sdm_residual_layer_norm_backward_workspace_bytes(int64_t rows, int64_t d) {
    return norm_backward_bytes(true, rows, d);
}

int sdm_residual_layer_norm_backward(const void* dy, const void* dh, int g_dtype, const void* h, int h_dtype,
                                     const float* gamma, float eps, int64_t rows, int64_t d, void* dx, float* dgamma,
                                     float* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    return norm_backward_impl("sdm_residual_layer_norm_backward", true, dy, dh, g_dtype, h, h_dtype, gamma, eps, rows, d,
                              dx, dgamma, dbias, workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace {

int check_balance(const char* fn, int64_t B, int64_t H, int64_t T, int64_t K, int64_t N) {
    if (B < 0 || H < 0 || T < 0 || K < 1 || N < 1) return fail(SDM_ERR_SHAPE, "%s: invalid sizes", fn);
    if (N > (1 << 18)) return fail(SDM_ERR_UNSUPPORTED, "%s: N=%lld: at most 2^18 slots", fn, (long long)N);
    if (K > 256) return fail(SDM_ERR_UNSUPPORTED, "%s: K=%lld: at most 256 slots a token", fn, (long long)K);
    // counts are 32-bit; each factor is bounded first, so that the products stay in 64 bits
    if (B > 0x7FFFFFFFll || H > 4096 || T > 0x7FFFFFFFll || B * T > 0x7FFFFFFFll || B * T * K > 0x7FFFFFFFll)
        return fail(SDM_ERR_UNSUPPORTED, "%s: at most 4096 heads, and 2^31 - 1 selections a head", fn);
    if (B * H > 0x7FFFFFFFll / 2 || B * H * (1 + T * K / sdm::BALANCE_PIECE) > 0x7FFFFFFFll)
        return fail(SDM_ERR_UNSUPPORTED, "%s: too many heads and sequences for one launch", fn);
    return 0;
}

}  // namespace

extern "C" {

int64_t sdm_balance_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t K, int64_t N) {
    if (check_balance("sdm_balance_workspace_bytes", B, H, T, K, N)) return -1;
    return H == 0 ? 0 : sdm::balance_workspace_bytes(B, H, T, K, N);
}

int sdm_balance_forward(const int32_t* idx, const float* wt, const uint8_t* mask, int64_t B, int64_t H, int64_t T,
                        int64_t K, int64_t N, int32_t* counts, float* mass, int32_t* tokens, float* loss,
                        void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_balance_forward";
    int rc = check_balance(fn, B, H, T, K, N);
    if (rc) return rc;
    if (H == 0) return ok();
    const bool some = B > 0 && T > 0;
    if (some && (rc = check_buffers(fn, {idx, wt}))) return rc;
    if ((rc = check_buffers(fn, {counts, mass, tokens, loss}))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, sdm::balance_workspace_bytes(B, H, T, K, N)))) return rc;
    sdm::BalanceArgs a{};
    a.idx = idx; a.wt = wt; a.mask = some ? mask : nullptr;
    a.counts = counts; a.mass = mass; a.tokens = tokens; a.loss = loss;
    a.B = B; a.H = H; a.T = T; a.K = K; a.N = N;
    a.workspace = workspace;
    hipError_t e = sdm::launch_balance(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

int sdm_balance_backward(const int32_t* idx, const uint8_t* mask, const int32_t* counts, const int32_t* tokens,
                         const float* dloss, int64_t B, int64_t H, int64_t T, int64_t K, int64_t N, float* dwt,
                         void* stream) {
    const char* fn = "sdm_balance_backward";
    int rc = check_balance(fn, B, H, T, K, N);
    if (rc) return rc;
    if (B == 0 || H == 0 || T == 0) return ok();
    if ((rc = check_buffers(fn, {idx, counts, tokens, dloss, dwt}))) return rc;
    sdm::BalanceBwdArgs a{};
    a.idx = idx; a.mask = mask; a.counts = counts; a.tokens = tokens; a.dloss = dloss; a.dwt = dwt;
    a.B = B; a.H = H; a.T = T; a.K = K; a.N = N;
    hipError_t e = sdm::launch_balance_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

}  // extern "C"

namespace {

constexpr int64_t MOST = 0x7FFFFFFFll;

// Strides (elements) of a tensor by strides: not negative, and its last element within 64 bits
int check_strides(const char* fn, const char* name, std::initializer_list<int64_t> sizes,
                  std::initializer_list<int64_t> strides) {
    __int128 last = 0;
    const int64_t* n = sizes.begin();
    for (int64_t s : strides) {
        if (s < 0) return fail(SDM_ERR_SHAPE, "%s: negative stride of %s", fn, name);
        last += (__int128)(*n > 0 ? *n - 1 : 0) * s;
        ++n;
    }
    return last < ((__int128)1 << 59) ? 0 : fail(SDM_ERR_UNSUPPORTED, "%s: strides of %s pass 64 bits", fn, name);
}

int check_address(const char* fn, const char* name, const void* p, int64_t bytes) {
    if (!p) return fail(SDM_ERR_NULL, "%s: %s is NULL", fn, name);
    return (uintptr_t)p % bytes == 0 ? 0 : fail(SDM_ERR_ALIGN, "%s: %s not aligned to its elements", fn, name);
}

// The largest power of two up to 8 elements that divides all of them (addresses in elements of `bytes`)
int common_align(std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> counts, int64_t bytes) {
    uint64_t all = 8;
    for (const void* p : ptrs) all |= p ? (uintptr_t)p / bytes : 0;
    for (int64_t n : counts) all |= (uint64_t)n;
    return (int)(all & (~all + 1));
}

int check_conv(const char* fn, int dtype, int act, int64_t B, int64_t H, int64_t T, int64_t d, int64_t K) {
    if (dtype != SDM_F32 && dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown dtype %d", fn, dtype);
    if (act != SDM_ACT_NONE && act != SDM_ACT_SILU) return fail(SDM_ERR_DTYPE, "%s: unknown activation %d", fn, act);
    if (B < 0 || H < 0 || T < 0 || d < 1 || K < 1) return fail(SDM_ERR_SHAPE, "%s: invalid sizes", fn);
    if (K < 2 || K > 8) return fail(SDM_ERR_UNSUPPORTED, "%s: K=%lld: from 2 to 8 taps", fn, (long long)K);
    // each factor below 2^31 first, so that the products stay in 64 bits
    const int64_t tiles = T > sdm::CONV_TILE_MIN ? (T + sdm::CONV_TILE_MIN - 1) / sdm::CONV_TILE_MIN : 1;
    if (B > MOST || H > MOST || T > MOST || d > MOST || H * d > 1 << 23 || B * tiles > MOST ||
        B * tiles * ((H * d + 63) / 64) >= 1 << 26)
        return fail(SDM_ERR_UNSUPPORTED, "%s: too many tokens and channels for one launch", fn);
    return B == 0 || H == 0 ? NO_WORK : 0;
}

// Rows by strides that a call writes: no element twice
int check_apart(const char* fn, const char* name, int64_t row, std::initializer_list<int64_t> sizes,
                std::initializer_list<int64_t> strides) {
    __int128 extent = row;  // of the dimensions so far, the nearest ones first
    bool used[3] = {};
    for (size_t k = 0; k < sizes.size(); ++k) {
        int at = -1;
        for (int i = 0; i < (int)sizes.size(); ++i)
            if (!used[i] && (at < 0 || strides.begin()[i] < strides.begin()[at])) at = i;
        used[at] = true;
        const int64_t n = sizes.begin()[at], s = strides.begin()[at];
        if (n <= 1) continue;
        if (s < extent) return fail(SDM_ERR_SHAPE, "%s: elements of %s share an address", fn, name);
        extent += (__int128)(n - 1) * s;
    }
    return 0;
}

}  // namespace

extern "C" {

int sdm_causal_conv_forward(const void* x, int dtype, const int64_t* x_strides, const float* w, const float* bias,
                            int act, const void* S0, void* S, const uint8_t* start, const int32_t* lengths, void* y,
                            int64_t B, int64_t H, int64_t T, int64_t d, int64_t K, void* stream) {
    const char* fn = "sdm_causal_conv_forward";
    int rc = check_conv(fn, dtype, act, B, H, T, d, K);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    const int64_t flat[3] = {H * T * d, T * d, d}, *xs = x_strides ? x_strides : flat, es = dtype == SDM_BF16 ? 2 : 4;
    if ((rc = check_strides(fn, "x", {B, H, T}, {xs[0], xs[1], xs[2]}))) return rc;
    if (T > 0 && ((rc = check_address(fn, "x", x, es)) || (rc = check_buffers(fn, {y})))) return rc;
    if ((rc = check_buffers(fn, {w}))) return rc;
    const void* opt[] = {bias, S0, S};
    for (const void* p : opt)
        if (p && !aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    if (lengths && (rc = check_address(fn, "lengths", lengths, 4))) return rc;
    if (T > 0 && (y == x || y == S0 || y == S)) return fail(SDM_ERR_SHAPE, "%s: y may not alias x, S0 or S", fn);
    if (T > 0 && (rc = check_own(fn, {S}, {x, w, bias}))) return rc;
    sdm::ConvArgs a{};
    a.x = x; a.w = w; a.bias = bias; a.S0 = S0; a.S = S; a.start = start; a.lengths = lengths; a.y = y;
    a.x_b = xs[0]; a.x_h = xs[1]; a.x_t = xs[2];
    a.B = B; a.H = H; a.T = T; a.d = (int)d; a.K = (int)K;
    a.align = common_align({x}, {d, xs[0], xs[1], xs[2]}, es);
    a.bf16 = dtype == SDM_BF16; a.silu = act == SDM_ACT_SILU;
    hipError_t e = sdm::launch_conv(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

int64_t sdm_causal_conv_backward_workspace_bytes(int64_t B, int64_t H, int64_t T, int64_t d, int64_t K) {
    const int rc = check_conv("sdm_causal_conv_backward_workspace_bytes", SDM_F32, SDM_ACT_NONE, B, H, T, d, K);
    if (rc == NO_WORK) return 0;
    return rc ? -1 : sdm::conv_backward_workspace_bytes(B, H, T, d, (int)K);
}

int sdm_causal_conv_backward(const void* dy, const void* x, int dtype, const int64_t* x_strides, const float* w,
                             const float* bias, int act, const void* S0, const void* dS, const uint8_t* start,
                             const int32_t* lengths, void* dx, const int64_t* dx_strides, float* dw, float* dbias,
                             void* dS0, int64_t B, int64_t H, int64_t T, int64_t d, int64_t K, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_causal_conv_backward";
    int rc = check_conv(fn, dtype, act, B, H, T, d, K);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    const int64_t flat[3] = {H * T * d, T * d, d}, es = dtype == SDM_BF16 ? 2 : 4;
    const int64_t *xs = x_strides ? x_strides : flat, *gs = dx_strides ? dx_strides : flat;
    if ((rc = check_strides(fn, "x", {B, H, T}, {xs[0], xs[1], xs[2]}))) return rc;
    if ((rc = check_strides(fn, "dx", {B, H, T}, {gs[0], gs[1], gs[2]}))) return rc;
    if (T > 0) {  // (of no tokens dx has no element, whatever its strides)
        if ((rc = check_apart(fn, "dx", d, {B, H, T}, {gs[0], gs[1], gs[2]}))) return rc;
        if ((rc = check_address(fn, "x", x, es)) || (rc = check_address(fn, "dx", dx, es)) || (rc = check_buffers(fn, {dy})))
            return rc;
        if (dx == x || dx == dy || (dS0 && (dS0 == dS || dS0 == S0 || dS0 == dx)))
            return fail(SDM_ERR_SHAPE, "%s: dx and dS0 may not alias an input or each other", fn);
    }
    if ((rc = check_buffers(fn, {w, dw}))) return rc;
    const void* opt[] = {bias, S0, dS, dbias, dS0};
    for (const void* p : opt)
        if (p && !aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    if (lengths && (rc = check_address(fn, "lengths", lengths, 4))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, sdm::conv_backward_workspace_bytes(B, H, T, d, (int)K)))) return rc;
    // dw and dbias are written behind the pass that reads the inputs; of no tokens only the states are looked at
    const void* tx = T > 0 ? dx : nullptr;
    if ((rc = check_own(fn, {tx, dS0, dw, dbias}, {})) || (T > 0 && (rc = check_own(fn, {tx, dS0}, {dy, x, w, bias, S0, dS})))) return rc;
    sdm::ConvBwdArgs a{};
    a.dy = dy; a.x = x; a.w = w; a.bias = bias; a.S0 = S0; a.dS = dS; a.start = start; a.lengths = lengths;
    a.dx = dx; a.dw = dw; a.dbias = dbias; a.dS0 = dS0;
    a.part = static_cast<float*>(workspace);
    a.x_b = xs[0]; a.x_h = xs[1]; a.x_t = xs[2];
    a.dx_b = gs[0]; a.dx_h = gs[1]; a.dx_t = gs[2];
    a.B = B; a.H = H; a.T = T; a.d = (int)d; a.K = (int)K;
    a.align = common_align({x, dx}, {d, xs[0], xs[1], xs[2], gs[0], gs[1], gs[2]}, es);
    a.bf16 = dtype == SDM_BF16; a.silu = act == SDM_ACT_SILU;
    hipError_t e = sdm::launch_conv_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

}  // extern "C"

namespace {

int check_selective(const char* fn, int in_dtype, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    if (in_dtype != SDM_F32 && in_dtype != SDM_BF16) return fail(SDM_ERR_DTYPE, "%s: unknown dtype %d", fn, in_dtype);
    if (B < 0 || T < 0 || D < 1 || G < 1 || N < 1 || D % G != 0)
        return fail(SDM_ERR_SHAPE, "%s: invalid sizes (G has to divide D)", fn);
    if (N > 64) return fail(SDM_ERR_UNSUPPORTED, "%s: N=%lld: at most 64 states a channel", fn, (long long)N);
    if (D > (1 << 20)) return fail(SDM_ERR_UNSUPPORTED, "%s: D=%lld: at most 2^20 channels", fn, (long long)D);
    // fewer than 2^32 threads a launch, 1024 a tile of 64 channels and 16 states; each factor is bounded first
    if (B > MOST || T > MOST || B * G >= 1 << 22 || sdm::sel_tiles(B, (int)G, (int)D) * ((N + 15) / 16) >= 1 << 22)
        return fail(SDM_ERR_UNSUPPORTED, "%s: too many sequences and channels for one launch", fn);
    return B == 0 ? NO_WORK : 0;
}
int check_selective_backward(const char* fn, int in_dtype, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const int rc = check_selective(fn, in_dtype, B, T, D, G, N);
    // fewer than 2^32 threads for the sums: 32 a token, group and tile of states, in workgroups of 256; 32768 a tile's gradient of A
    if (rc == 0 && (B * G * T * ((N + 15) / 16) > (1 << 27) - 8 || sdm::sel_tiles(1, (int)G, (int)D) * ((N + 15) / 16) >= 1 << 17))
        return fail(SDM_ERR_UNSUPPORTED, "%s: too many tokens or groups for one launch", fn);
    return rc;
}

struct SelTensor {
    const char* name;
    const void* p;
    const int64_t* s;  // batch, token (group)
    bool bc;
};
int check_selective_tensors(const char* fn, std::initializer_list<SelTensor> ts, int64_t es, int64_t B, int64_t T, int64_t G) {
    int rc;
    for (const SelTensor& t : ts) {
        if (T > 0 && (rc = check_address(fn, t.name, t.p, es))) return rc;
        rc = t.bc ? check_strides(fn, t.name, {B, T, G}, {t.s[0], t.s[1], t.s[2]}) : check_strides(fn, t.name, {B, T}, {t.s[0], t.s[1]});
        if (rc) return rc;
        if (t.s[1] >= 1 << 26)  // a chunk's rows lie within 2^31 bytes
            return fail(SDM_ERR_UNSUPPORTED, "%s: token stride of %s: below 2^26 elements", fn, t.name);
    }
    return 0;
}

template <typename Args>
void selective_args(Args& a, const void* x, const void* dt, const void* z, const void* Bm, const void* Cm, int in_dtype,
                    const int64_t* s, const float* A, const float* Dskip, const float* dt_bias, int softplus,
                    const float* S0, const uint8_t* start, const int32_t* lengths, int64_t B, int64_t T, int64_t D,
                    int64_t G, int64_t N, void* workspace) {
    a.x = x; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm; a.bf16 = in_dtype == SDM_BF16;
    a.x_b = s[0]; a.x_t = s[1]; a.dt_b = s[2]; a.dt_t = s[3]; a.z_b = s[4]; a.z_t = s[5];
    a.B_b = s[6]; a.B_t = s[7]; a.B_g = s[8]; a.C_b = s[9]; a.C_t = s[10]; a.C_g = s[11];
    a.A = A; a.Dskip = Dskip; a.bias = dt_bias; a.softplus = softplus != 0; a.S0 = S0;
    a.start = start; a.lengths = lengths;
    a.B = B; a.T = T; a.D = (int)D; a.G = (int)G; a.N = (int)N;
    a.workspace = workspace;
}

}  // namespace

extern "C" {

int64_t sdm_selective_scan_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const int rc = check_selective("sdm_selective_scan_workspace_bytes", SDM_F32, B, T, D, G, N);
    if (rc == NO_WORK) return 0;
    return rc ? -1 : sdm::selective_workspace_bytes(B, T, (int)G, (int)D, (int)N);
}

int sdm_selective_scan_forward(const void* x, const void* dt, const void* z, const void* Bm, const void* Cm,
                               int in_dtype, const int64_t* strides, const float* A, const float* Dskip,
                               const float* dt_bias, int softplus, const float* S0, float* S, const uint8_t* start,
                               const int32_t* lengths, void* y, int64_t B, int64_t T, int64_t D, int64_t G, int64_t N,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_selective_scan_forward";
    int rc = check_selective(fn, in_dtype, B, T, D, G, N);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    const int64_t td = T * D, tg = T * G * N, gn = G * N, es = in_dtype == SDM_BF16 ? 2 : 4;
    const int64_t flat[12] = {td, D, td, D, td, D, tg, gn, N, tg, gn, N}, *s = strides ? strides : flat;
    if ((rc = check_selective_tensors(fn, {{"x", x, s, false}, {"dt", dt, s + 2, false}, {"Bm", Bm, s + 6, true}, {"Cm", Cm, s + 9, true}},
                                      es, B, T, G)))
        return rc;
    if (z && (rc = check_selective_tensors(fn, {{"z", z, s + 4, false}}, es, B, T, G))) return rc;
    if ((rc = check_buffers(fn, {A})) || (T > 0 && (rc = check_buffers(fn, {y})))) return rc;
    const void* opt[] = {Dskip, dt_bias, S0, S};
    for (const void* p : opt)
        if (p && !aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    if (lengths && (rc = check_address(fn, "lengths", lengths, 4))) return rc;
    if (T > 0 && (y == x || y == dt || y == z || y == Bm || y == Cm || y == S0 || y == S))
        return fail(SDM_ERR_SHAPE, "%s: y may not alias an input or S", fn);
    const int64_t need = sdm::selective_workspace_bytes(B, T, (int)G, (int)D, (int)N);
    if (need > 0 && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
    if (T > 0 && (rc = check_own(fn, {S}, {x, dt, z, Bm, Cm, A, Dskip, dt_bias}))) return rc;
    sdm::SelArgs a{};
    selective_args(a, x, dt, z, Bm, Cm, in_dtype, s, A, Dskip, dt_bias, softplus, S0, start, lengths, B, T, D, G, N, workspace);
    a.S = S; a.y = y;
    hipError_t e = sdm::launch_selective(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

int64_t sdm_selective_scan_backward_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t G, int64_t N) {
    const int rc = check_selective_backward("sdm_selective_scan_backward_workspace_bytes", SDM_F32, B, T, D, G, N);
    if (rc == NO_WORK) return 0;
    return rc ? -1 : sdm::selective_backward_workspace_bytes(B, T, (int)G, (int)D, (int)N);
}

int sdm_selective_scan_backward(const void* dy, const void* x, const void* dt, const void* z, const void* Bm,
                                const void* Cm, int in_dtype, const int64_t* strides, const float* A,
                                const float* Dskip, const float* dt_bias, int softplus, const float* S0,
                                const float* dS, const uint8_t* start, const int32_t* lengths, void* dx, void* ddt,
                                void* dz, float* dA, float* dB, float* dC, float* dD, float* ddt_bias, float* dS0,
                                int64_t B, int64_t T, int64_t D, int64_t G, int64_t N, void* workspace,
                                int64_t workspace_bytes, void* stream) {
    const char* fn = "sdm_selective_scan_backward";
    int rc = check_selective_backward(fn, in_dtype, B, T, D, G, N);
    if (rc == NO_WORK) return ok();
    if (rc) return rc;
    const int64_t td = T * D, tg = T * G * N, gn = G * N, es = in_dtype == SDM_BF16 ? 2 : 4;
    const int64_t flat[14] = {td, D, td, D, td, D, tg, gn, N, tg, gn, N, td, D}, *s = strides ? strides : flat;
    if ((rc = check_selective_tensors(fn, {{"x", x, s, false}, {"dt", dt, s + 2, false}, {"Bm", Bm, s + 6, true}, {"Cm", Cm, s + 9, true},
                                           {"dy", dy, s + 12, false}}, es, B, T, G)))
        return rc;
    if (z && (rc = check_selective_tensors(fn, {{"z", z, s + 4, false}}, es, B, T, G))) return rc;
    if ((rc = check_buffers(fn, {A, dA}))) return rc;
    if (T > 0 && ((rc = check_buffers(fn, {dx, ddt, dB, dC})) || (z && (rc = check_buffers(fn, {dz}))))) return rc;
    const void* opt[] = {Dskip, dt_bias, S0, dS, dD, ddt_bias, dS0};
    for (const void* p : opt)
        if (p && !aligned16(p)) return fail(SDM_ERR_ALIGN, "%s: pointer %p not 16-byte aligned", fn, p);
    if (lengths && (rc = check_address(fn, "lengths", lengths, 4))) return rc;
    if (T > 0) {
        const void *outs[] = {dx, ddt, z ? dz : nullptr, dB, dC}, *ins[] = {x, dt, z, Bm, Cm, dy, S0, dS};
        for (const void* o : outs)
            for (const void* i : ins)
                if (o && o == i) return fail(SDM_ERR_SHAPE, "%s: a gradient may not alias an input", fn);
    }
    if ((rc = check_workspace(workspace, workspace_bytes,
                              sdm::selective_backward_workspace_bytes(B, T, (int)G, (int)D, (int)N))))
        return rc;
    // dA, dD and ddt_bias are written behind the last pass, which reads all inputs but S0 and dS
    const bool any = T > 0;
    const void *tx = any ? dx : nullptr, *tdt = any ? ddt : nullptr, *tz = any && z ? dz : nullptr, *tB = any ? dB : nullptr, *tC = any ? dC : nullptr;
    if ((rc = check_own(fn, {tx, tdt, tz, tB, tC, dS0, dA, dD, ddt_bias}, {})) ||
        (any && (rc = check_own(fn, {tx, tdt, tz, tB, tC, dS0}, {dy, x, dt, z, Bm, Cm, A, Dskip, dt_bias}))))
        return rc;
    sdm::SelBwdArgs a{};
    selective_args(a, x, dt, z, Bm, Cm, in_dtype, s, A, Dskip, dt_bias, softplus, S0, start, lengths, B, T, D, G, N, workspace);
    a.dy = dy; a.dS = dS; a.dy_b = s[12]; a.dy_t = s[13];
    a.dx = dx; a.ddt = ddt; a.dz = z ? dz : nullptr; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dbias = ddt_bias; a.dS0 = dS0;
    hipError_t e = sdm::launch_selective_backward(a, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ok() : hip_fail(e, fn);
}

}  // extern "C"
