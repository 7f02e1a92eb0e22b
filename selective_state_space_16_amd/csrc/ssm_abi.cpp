// C ABI of libssm.so: argument checks on the host, then kernel dispatch.
// Every check runs before any HIP call, so a rejected call launches nothing.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "../../include/ssm.h"
#include "ssm_internal.h"

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 46;  // keeps every byte offset far from overflow

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

bool supported_n(int64_t N) { return N == 1 || N == 2 || N == 4 || N == 8 || N == 16; }

// Product of non-negative sizes, or -1 when it exceeds kMaxElems.
int64_t checked_mul(int64_t a, int64_t b) {
    if (a == 0 || b == 0) return 0;
    if (a > kMaxElems / b) return -1;
    return a * b;
}

int64_t checked_mul3(int64_t a, int64_t b, int64_t c) {
    const int64_t ab = checked_mul(a, b);
    return ab < 0 ? -1 : checked_mul(ab, c);
}

size_t round_up256(size_t n) { return (n + 255) / 256 * 256; }

// Both scans keep a header of ssm::kHdrBytes at the start of the workspace
// (its words are described in ssm_internal.h); the chunked scan leaves it alone.
constexpr size_t kHeader = ssm::kHdrBytes;

// Workspace of the chunked three-launch scan:
// [header | chunk states (batch,K,D,N) | summed deltas (batch,K,D)].
size_t twopass_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t *K, int64_t *Lc) {
    ssm::scan_plan(batch, L, D, N, K, Lc);
    if (*K <= 1) return 0;
    return kHeader + round_up256((size_t)batch * *K * D * N * sizeof(float)) +
           round_up256((size_t)batch * *K * D * sizeof(float));
}

// Workspace of the stripe scan.
size_t stripe_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype, ssm::StripePlan *p) {
    if (!ssm::stripe_plan(batch, L, D, N, dtype, p)) return 0;
    return p->bytes;
}

// Which scan runs. The stripe scan reads 16-byte pieces of channel rows and
// Bt/Ct rows; shapes it cannot take run the chunked three-launch scan, which
// SSM_SCAN_IMPL=twopass also selects (for comparison).
enum class Impl { kTwopass, kStripe };

Impl choose_impl(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    ssm::StripePlan sp;
    const bool stripe_ok = ssm::stripe_plan(batch, L, D, N, dtype, &sp) && sp.supported;
    const char *e = getenv("SSM_SCAN_IMPL");
    if (e && strcmp(e, "twopass") == 0) return Impl::kTwopass;
    return stripe_ok ? Impl::kStripe : Impl::kTwopass;
}

// Whether cut stripes take early mode: by their length, or as
// SSM_STRIPE_EARLY=0/1 says (for comparison and tests).
int stripe_early(const ssm::StripePlan &p) {
    const char *e = getenv("SSM_STRIPE_EARLY");
    if (e && (strcmp(e, "0") == 0 || strcmp(e, "1") == 0)) return e[0] == '1';
    return p.early ? 1 : 0;
}

size_t workspace_for(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    int64_t K, Lc;
    ssm::StripePlan sp;
    return choose_impl(batch, L, D, N, dtype) == Impl::kStripe ? stripe_workspace(batch, L, D, N, dtype, &sp)
                                                               : twopass_workspace(batch, L, D, N, &K, &Lc);
}

constexpr int64_t kMaxNorm = ((int64_t)1 << 28) - 64;  // channels that one launch of the gradients' reduction reaches
constexpr int64_t kMaxRow = (int64_t)1 << 23;  // elements between rows of the cache entry points' inputs

// Sizes the SSD layer on a cache takes: heads of 64 to 256 in whole 64s, N of
// 64 or 128, rows and sequences that the kernels' offsets and grids reach.
bool ssd_cache_sizes(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N) {
    if (P < 64 || P > 256 || P % 64 != 0 || (N != 64 && N != 128)) return false;
    if (seqs > 65535 || rows > INT32_MAX || H >= kMaxRow / P || G >= kMaxRow / (2 * N)) return false;
    const int64_t C = H * P + 2 * G * N, chunks = rows / 64 + seqs;
    // threads of a launch: per chunk of 64 tokens (or request) and group, 16
    // heads, or 64 rows of a head's state
    return C < kMaxRow && (chunks * (G + H / 16 + 1) + seqs * (C / 512 + 1)) * 1024 <= UINT32_MAX &&
           chunks * (H * P / 64 * 256 + G * 512) <= UINT32_MAX;
}

// Floats per request in the step's workspace: x | B | C, dt and exp(dt A),
// in whole 16-byte pieces.
int64_t ssd_step_row(int64_t H, int64_t P, int64_t G, int64_t N) { return (H * P + 2 * G * N + 2 * H + 3) / 4 * 4; }

}  // namespace

extern "C" {

const char *ssm_status_string(int status) {
    switch (status) {
        case SSM_OK: return "ok";
        case SSM_ERR_NULL: return "a required pointer is NULL";
        case SSM_ERR_SHAPE: return "a size is negative or the tensor sizes overflow";
        case SSM_ERR_DTYPE: return "dtype must be SSM_F32 or SSM_BF16";
        case SSM_ERR_UNSUPPORTED: return "N (1, 2, 4, 8 or 16 in a selective scan) or another size is not one this entry point supports";
        case SSM_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case SSM_ERR_WORKSPACE: return "workspace is missing or too small";
        case SSM_ERR_HIP: return "a HIP launch failed";
        case SSM_ERR_TIMEOUT: return "a wait for another workgroup's results gave up; the outputs that depend on them are NaN";
        default: return "unknown status";
    }
}

const char *ssm_version(void) { return "ssm-gfx950 0.1"; }

int ssm_scan_workspace_status(const void *workspace, size_t workspace_bytes, void *stream) {
    if (!workspace || workspace_bytes < kHeader) return SSM_OK;  // no header: nothing can have failed
    if (!aligned16(workspace)) return SSM_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    uint32_t hdr[4] = {0, 0, 0, 0};
    if (hipMemcpyAsync(hdr, workspace, sizeof(hdr), hipMemcpyDeviceToHost, s) != hipSuccess) return SSM_ERR_HIP;
    if (hipStreamSynchronize(s) != hipSuccess) return SSM_ERR_HIP;
    // the last call failed when the error word carries its tag
    return hdr[ssm::kHdrError] != 0 && hdr[ssm::kHdrError] == hdr[ssm::kHdrEpoch] ? SSM_ERR_TIMEOUT : SSM_OK;
}

size_t ssm_scan_workspace_bytes(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    if (batch < 0 || L < 0 || D < 0 || !supported_n(N)) return 0;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return 0;
    if (checked_mul3(batch, L, D) < 0 || checked_mul3(batch, D, N) < 0) return 0;
    if (batch == 0 || L == 0 || D == 0) return 0;
    return workspace_for(batch, L, D, N, dtype);
}

// Extra inputs of the exponential-trapezoidal rule: the per-token weight and
// the token before the first (both of x_prev and B_prev, or neither); and of
// the x branch ahead of the scan: the taps, bias and earlier raw x of its
// convolution (conv_w NULL: x is used as given).
struct TrapIn {
    const void *lam = nullptr, *x_prev = nullptr, *B_prev = nullptr;
    const float *conv_w = nullptr, *conv_b = nullptr;
    const void *conv_state = nullptr;
};

static int scan_fwd(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                    const void *x, const void *delta, const float *dt_bias, int softplus, const float *A,
                    const void *Bt, const void *Ct, const float *Dskip,
                    const void *z, const float *state_in, float *state_out,
                    void *y, void *workspace, size_t workspace_bytes, void *stream, TrapIn tr = {},
                    bool launch = true) {
    // launch = false: check the arguments only (every check below precedes
    // the first HIP call)
    if (batch < 0 || L < 0 || D < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!supported_n(N)) return SSM_ERR_UNSUPPORTED;
    if (checked_mul3(batch, L, D) < 0 || checked_mul3(batch, L, N) < 0 || checked_mul3(batch, D, N) < 0)
        return SSM_ERR_SHAPE;
    if (batch == 0 || D == 0) return SSM_OK;
    hipStream_t s = (hipStream_t)stream;
    if (L == 0) {
        if (!state_out) return SSM_OK;
        if (!aligned16(state_out) || (state_in && !aligned16(state_in))) return SSM_ERR_ALIGN;
        if (state_in == state_out || !launch) return SSM_OK;
        return ssm::launch_state_copy(state_in, state_out, batch * D * N, s) == hipSuccess ? SSM_OK
                                                                                          : SSM_ERR_HIP;
    }
    if (!x || !delta || !A || !Bt || !Ct || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bt, Ct, Dskip, z, state_in, state_out, y, dt_bias, tr.lam, tr.x_prev,
                          tr.B_prev, tr.conv_w, tr.conv_b, tr.conv_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;

    const size_t need = workspace_for(batch, L, D, N, dtype);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
        if (!aligned16(workspace)) return SSM_ERR_ALIGN;
    }
    if (!launch) return SSM_OK;
    const Impl impl = choose_impl(batch, L, D, N, dtype);
    if (impl == Impl::kStripe) {
        ssm::StripePlan p;
        stripe_workspace(batch, L, D, N, dtype, &p);
        ssm::StripeArgs a{};
        a.batch = batch;
        a.L = L;
        a.D = D;
        a.x = x;
        a.delta = delta;
        a.Bt = Bt;
        a.Ct = Ct;
        a.z = z;
        a.A = A;
        a.Dskip = Dskip;
        a.state_in = state_in;
        a.state_out = state_out;
        a.dt_bias = dt_bias;
        a.delta_softplus = softplus;
        a.lam = tr.lam;
        a.x_prev = tr.x_prev;
        a.B_prev = tr.B_prev;
        a.conv_w = tr.conv_w;
        a.conv_b = tr.conv_b;
        a.conv_state = tr.conv_state;
        a.y = y;
        a.ntpb = p.ntpb;
        a.ncol = p.ncol;
        a.cols_per_list = p.cols_per_list;
        a.n_whole = p.n_whole;
        a.S = p.S;
        a.SL = p.SL;
        a.early = stripe_early(p);
        char *w = (char *)workspace;
        a.hdr = (uint32_t *)w;
        a.incl = (uint64_t *)(w + p.off_incl);
        a.agg = (uint64_t *)(w + p.off_agg);
        return ssm::launch_scan_stripe(a, (int)N, dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
    ssm::ScanArgs a{};
    a.batch = batch;
    a.L = L;
    a.D = D;
    a.x = x;
    a.delta = delta;
    a.Bt = Bt;
    a.Ct = Ct;
    a.z = z;
    a.A = A;
    a.Dskip = Dskip;
    a.state_in = state_in;
    a.dt_bias = dt_bias;
    a.delta_softplus = softplus;
    a.lam = tr.lam;
    a.x_prev = tr.x_prev;
    a.B_prev = tr.B_prev;
    a.conv_w = tr.conv_w;
    a.conv_b = tr.conv_b;
    a.conv_state = tr.conv_state;
    a.state_out = state_out;
    a.y = y;
    if (twopass_workspace(batch, L, D, N, &a.K, &a.Lc) > 0) {
        char *w = (char *)workspace + kHeader;
        a.ws_state = (float *)w;
        a.ws_dsum = (float *)(w + round_up256((size_t)batch * a.K * D * N * sizeof(float)));
    }
    return ssm::launch_scan(a, (int)N, dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

static int step(int64_t batch, int64_t D, int64_t N, int dtype,
                const void *x, const void *delta, const float *dt_bias, int softplus, const float *A,
                const void *Bt, const void *Ct, const float *Dskip,
                const void *z, float *state, void *y, void *stream, TrapIn tr = {}) {
    if (batch < 0 || D < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!supported_n(N)) return SSM_ERR_UNSUPPORTED;
    if (checked_mul3(batch, D, N) < 0) return SSM_ERR_SHAPE;
    if (batch == 0 || D == 0) return SSM_OK;
    if (!x || !delta || !A || !Bt || !Ct || !state || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bt, Ct, Dskip, z, state, y, dt_bias, tr.lam, tr.x_prev, tr.B_prev,
                          tr.conv_w, tr.conv_b, tr.conv_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::StepArgs a{};
    a.batch = batch;
    a.D = D;
    a.x = x;
    a.delta = delta;
    a.Bt = Bt;
    a.Ct = Ct;
    a.z = z;
    a.A = A;
    a.Dskip = Dskip;
    a.state = state;
    a.y = y;
    a.dt_bias = dt_bias;
    a.delta_softplus = softplus;
    a.lam = tr.lam;
    a.x_prev = tr.x_prev;
    a.B_prev = tr.B_prev;
    a.conv_w = tr.conv_w;
    a.conv_b = tr.conv_b;
    a.conv_state = const_cast<void *>(tr.conv_state);
    return ssm::launch_step(a, (int)N, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_scan_fwd(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                 const void *x, const void *delta, const float *A,
                 const void *Bt, const void *Ct, const float *Dskip,
                 const void *z, const float *state_in, float *state_out,
                 void *y, void *workspace, size_t workspace_bytes, void *stream) {
    return scan_fwd(batch, L, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state_in, state_out, y,
                    workspace, workspace_bytes, stream);
}

int ssm_scan_fwd_dt(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                    const void *x, const void *delta_raw, const float *dt_bias, const float *A,
                    const void *Bt, const void *Ct, const float *Dskip,
                    const void *z, const float *state_in, float *state_out,
                    void *y, void *workspace, size_t workspace_bytes, void *stream) {
    return scan_fwd(batch, L, D, N, dtype, x, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip, z, state_in, state_out, y,
                    workspace, workspace_bytes, stream);
}

int ssm_scan_fwd_conv(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                      const void *x_raw, const float *conv_w, const float *conv_b, const void *conv_state,
                      const void *delta_raw, const float *dt_bias, const float *A,
                      const void *Bt, const void *Ct, const float *Dskip,
                      const void *z, const float *state_in, float *state_out,
                      void *y, void *workspace, size_t workspace_bytes, void *stream) {
    if (!conv_w && batch > 0 && L > 0 && D > 0) return SSM_ERR_NULL;
    TrapIn tr;
    tr.conv_w = conv_w;
    tr.conv_b = conv_b;
    tr.conv_state = conv_state;
    return scan_fwd(batch, L, D, N, dtype, x_raw, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip, z, state_in, state_out,
                    y, workspace, workspace_bytes, stream, tr);
}

int ssm_scan_fwd_trap(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                      const void *x, const void *delta, const void *lam, const float *A,
                      const void *Bt, const void *Ct, const float *Dskip, const void *z,
                      const void *x_prev, const void *B_prev, const float *state_in, float *state_out,
                      void *y, void *workspace, size_t workspace_bytes, void *stream) {
    if (!lam && batch > 0 && L > 0 && D > 0) return SSM_ERR_NULL;
    if ((x_prev == nullptr) != (B_prev == nullptr)) return SSM_ERR_NULL;
    TrapIn tr;
    tr.lam = lam;
    tr.x_prev = x_prev;
    tr.B_prev = B_prev;
    return scan_fwd(batch, L, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state_in, state_out, y,
                    workspace, workspace_bytes, stream, tr);
}

int ssm_step(int64_t batch, int64_t D, int64_t N, int dtype,
             const void *x, const void *delta, const float *A,
             const void *Bt, const void *Ct, const float *Dskip,
             const void *z, float *state, void *y, void *stream) {
    return step(batch, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state, y, stream);
}

int ssm_step_dt(int64_t batch, int64_t D, int64_t N, int dtype,
                const void *x, const void *delta_raw, const float *dt_bias, const float *A,
                const void *Bt, const void *Ct, const float *Dskip,
                const void *z, float *state, void *y, void *stream) {
    return step(batch, D, N, dtype, x, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip, z, state, y, stream);
}

int ssm_step_conv(int64_t batch, int64_t D, int64_t N, int dtype,
                  const void *x_raw, const float *conv_w, const float *conv_b, void *conv_state,
                  const void *delta_raw, const float *dt_bias, const float *A,
                  const void *Bt, const void *Ct, const float *Dskip,
                  const void *z, float *state, void *y, void *stream) {
    if ((!conv_w || !conv_state) && batch > 0 && D > 0) return SSM_ERR_NULL;
    TrapIn tr;
    tr.conv_w = conv_w;
    tr.conv_b = conv_b;
    tr.conv_state = conv_state;
    return step(batch, D, N, dtype, x_raw, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip, z, state, y, stream, tr);
}

int ssm_step_trap(int64_t batch, int64_t D, int64_t N, int dtype,
                  const void *x, const void *delta, const void *lam, const float *A,
                  const void *Bt, const void *Ct, const float *Dskip, const void *z,
                  const void *x_prev, const void *B_prev, float *state, void *y, void *stream) {
    if (!lam && batch > 0 && D > 0) return SSM_ERR_NULL;
    if ((x_prev == nullptr) != (B_prev == nullptr)) return SSM_ERR_NULL;
    TrapIn tr;
    tr.lam = lam;
    tr.x_prev = x_prev;
    tr.B_prev = B_prev;
    return step(batch, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state, y, stream, tr);
}

// Workspace of the gradient: [header | hst | dsum | gq | pdB | pdC | pdA | pdD | pdT | pdBp | ckp | ckd].
struct BwdLayout {
    int64_t K;
    size_t off[11], bytes;
};

static BwdLayout bwd_layout(int64_t batch, int64_t L, int64_t D, int64_t N) {
    BwdLayout w{};
    w.K = (L + ssm::kBwdChunk - 1) / ssm::kBwdChunk;
    const int64_t nDB = ssm::bwd_channel_blocks(D, N, true);  // the most blocks: the trapezoidal rule
    const size_t sz[11] = {(size_t)(batch * w.K * D * N), (size_t)(batch * w.K * D), (size_t)(batch * w.K * D * N),
                           (size_t)(nDB * batch * L * N), (size_t)(nDB * batch * L * N),
                           (size_t)(batch * w.K * D * N), (size_t)(batch * w.K * D), (size_t)(batch * w.K * D),
                           (size_t)(nDB * batch * N), (size_t)(batch * w.K * ssm::kBwdCk * D * N),
                           (size_t)(batch * w.K * ssm::kBwdCk * D)};
    size_t off = kHeader;
    for (int i = 0; i < 11; ++i) {
        w.off[i] = off;
        off += round_up256(sz[i] * sizeof(float));
    }
    w.bytes = off;
    return w;
}

// Sizes the gradient accepts: every count within kMaxElems and every flat
// grid within 2^32 work-items.
static bool bwd_sizes_ok(int64_t batch, int64_t L, int64_t D, int64_t N) {
    const int64_t K = (L + ssm::kBwdChunk - 1) / ssm::kBwdChunk;
    if (checked_mul3(batch, L, D) < 0 || checked_mul3(batch, L, N) < 0 || checked_mul3(batch, D, N) < 0)
        return false;
    const int64_t nDB = ssm::bwd_channel_blocks(D, N, true);  // the most blocks: the trapezoidal rule
    if (checked_mul3(checked_mul(batch, K), D, N) < 0 || checked_mul3(checked_mul(nDB, batch), L, N) < 0)
        return false;
    const int64_t blocks = checked_mul3(nDB, K, batch);
    // the flat grids of the chunk kernels, the carry (batch * D * N lanes)
    // and the sums of dBt, dCt (batch * L * N lanes), in 256-lane blocks
    const int64_t lanes = checked_mul3(batch, D, N) > checked_mul3(batch, L, N) ? checked_mul3(batch, D, N)
                                                                                : checked_mul3(batch, L, N);
    return blocks >= 0 && blocks < ((int64_t)1 << 24) && lanes / 256 < ((int64_t)1 << 31);
}

size_t ssm_scan_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    if (batch <= 0 || L <= 0 || D <= 0 || !supported_n(N)) return 0;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return 0;
    if (!bwd_sizes_ok(batch, L, D, N)) return 0;
    return bwd_layout(batch, L, D, N).bytes;
}

// The gradient, for a step size given after its activation (softplus = 0) or
// before it (softplus = 1: delta holds delta_raw, ddelta receives its
// gradient, and ddt_bias, when given, the gradient of dt_bias).
// The trapezoidal rule's extra inputs and outputs.
struct TrapBwd {
    const void *lam = nullptr, *x_prev = nullptr, *B_prev = nullptr;
    void *dlam = nullptr, *dx_prev = nullptr;
    float *dB_prev = nullptr;
};

static int scan_bwd(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                    const void *x, const void *delta, const float *dt_bias, int softplus, const float *A,
                    const void *Bt, const void *Ct, const float *Dskip, const void *z, const float *state_in,
                    const void *dy, const float *dstate,
                    void *dx, void *ddelta, float *ddt_bias, float *dA, float *dBt, float *dCt, float *dDskip,
                    void *dz, float *dstate_in, void *workspace, size_t workspace_bytes, void *stream,
                    TrapBwd tr = {}, bool launch = true) {
    // launch = false: check the arguments only (every check below precedes
    // the first HIP call)
    if (batch < 0 || L < 0 || D < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!supported_n(N)) return SSM_ERR_UNSUPPORTED;
    if (!bwd_sizes_ok(batch, L, D, N)) return SSM_ERR_SHAPE;
    if (D > 0 && !dA) return SSM_ERR_NULL;
    if (z && !dz) return SSM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bt, Ct, Dskip, z, state_in, dy, dstate, dx, ddelta,
                          dA, dBt, dCt, dDskip, dz, dstate_in, workspace, dt_bias, ddt_bias,
                          tr.lam, tr.x_prev, tr.B_prev, tr.dlam, tr.dx_prev, tr.dB_prev};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    if (D == 0) return SSM_OK;
    if (batch == 0 || L == 0) {
        if (!launch) return SSM_OK;
        // nothing flows through the tokens: the parameter gradients are zero
        // and the gradient of the entering state is that of the leaving one
        if (ssm::launch_state_copy(nullptr, dA, D * N, s) != hipSuccess) return SSM_ERR_HIP;
        if (Dskip && dDskip && ssm::launch_state_copy(nullptr, dDskip, D, s) != hipSuccess) return SSM_ERR_HIP;
        if (ddt_bias && ssm::launch_state_copy(nullptr, ddt_bias, D, s) != hipSuccess) return SSM_ERR_HIP;

        if (dstate_in && dstate_in != dstate &&
            ssm::launch_state_copy(dstate, dstate_in, batch * D * N, s) != hipSuccess)
            return SSM_ERR_HIP;
        return SSM_OK;
    }
    if (!x || !delta || !A || !Bt || !Ct || !dy || !dx || !ddelta || !dBt || !dCt) return SSM_ERR_NULL;
    if (tr.lam && !tr.dlam) return SSM_ERR_NULL;
    const BwdLayout w = bwd_layout(batch, L, D, N);
    if (!workspace || workspace_bytes < w.bytes) return SSM_ERR_WORKSPACE;
    char *ws = (char *)workspace;
    ssm::BwdArgs a{};
    a.batch = batch;
    a.L = L;
    a.D = D;
    a.K = w.K;
    a.x = x;
    a.delta = delta;
    a.Bt = Bt;
    a.Ct = Ct;
    a.z = z;
    a.dy = dy;
    a.A = A;
    a.Dskip = Dskip;
    a.state_in = state_in;
    a.dstate = dstate;
    a.dx = dx;
    a.ddelta = ddelta;
    a.dz = dz;
    a.dA = dA;
    a.dBt = dBt;
    a.dCt = dCt;
    a.dDskip = Dskip ? dDskip : nullptr;
    a.dstate_in = dstate_in;
    a.dt_bias = dt_bias;
    a.delta_softplus = softplus;
    a.ddt_bias = softplus ? ddt_bias : nullptr;
    a.lam = tr.lam;
    a.x_prev = tr.x_prev;
    a.B_prev = tr.B_prev;
    a.dlam = tr.dlam;
    // the token before the first gets a gradient only when it is given, and
    // both of its outputs are asked for
    const bool prev_grad = tr.x_prev && tr.dx_prev && tr.dB_prev;
    a.dx_prev = prev_grad ? tr.dx_prev : nullptr;
    a.dB_prev = prev_grad ? tr.dB_prev : nullptr;
    a.hst = (float *)(ws + w.off[0]);
    a.dsum = (float *)(ws + w.off[1]);
    a.gq = (float *)(ws + w.off[2]);
    a.pdB = (float *)(ws + w.off[3]);
    a.pdC = (float *)(ws + w.off[4]);
    a.pdA = (float *)(ws + w.off[5]);
    a.pdD = (float *)(ws + w.off[6]);
    a.pdT = (float *)(ws + w.off[7]);
    a.pdBp = (float *)(ws + w.off[8]);
    a.ckp = (float *)(ws + w.off[9]);
    a.ckd = (float *)(ws + w.off[10]);
    if (!launch) return SSM_OK;
    return ssm::launch_scan_bwd(a, (int)N, dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_scan_bwd(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                 const void *x, const void *delta, const float *A, const void *Bt, const void *Ct,
                 const float *Dskip, const void *z, const float *state_in,
                 const void *dy, const float *dstate,
                 void *dx, void *ddelta, float *dA, float *dBt, float *dCt, float *dDskip, void *dz,
                 float *dstate_in, void *workspace, size_t workspace_bytes, void *stream) {
    return scan_bwd(batch, L, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state_in, dy, dstate, dx,
                    ddelta, nullptr, dA, dBt, dCt, dDskip, dz, dstate_in, workspace, workspace_bytes, stream);
}

int ssm_scan_bwd_trap(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                      const void *x, const void *delta, const void *lam, const float *A,
                      const void *Bt, const void *Ct, const float *Dskip, const void *z,
                      const void *x_prev, const void *B_prev, const float *state_in,
                      const void *dy, const float *dstate,
                      void *dx, void *ddelta, void *dlam, float *dA, float *dBt, float *dCt, float *dDskip, void *dz,
                      void *dx_prev, float *dB_prev, float *dstate_in, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (!lam && batch > 0 && L > 0 && D > 0) return SSM_ERR_NULL;
    if ((x_prev == nullptr) != (B_prev == nullptr)) return SSM_ERR_NULL;
    if ((dx_prev == nullptr) != (dB_prev == nullptr)) return SSM_ERR_NULL;
    TrapBwd tr;
    tr.lam = lam;
    tr.x_prev = x_prev;
    tr.B_prev = B_prev;
    tr.dlam = dlam;
    tr.dx_prev = dx_prev;
    tr.dB_prev = dB_prev;
    return scan_bwd(batch, L, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state_in, dy, dstate, dx,
                    ddelta, nullptr, dA, dBt, dCt, dDskip, dz, dstate_in, workspace, workspace_bytes, stream, tr);
}

// Workspace of the gradient through the x branch: the scan gradient's, then
// the branch's output and its gradient (activation dtype) and the partial
// sums of the taps' and bias' gradients.
struct ConvBwdLayout {
    int64_t chunk, nchunk;
    size_t bwd, off_xc, off_gx, off_part, bytes;
};

static ConvBwdLayout conv_bwd_layout(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    ConvBwdLayout w{};
    ssm::conv_bwd_plan(batch, L, D, &w.chunk, &w.nchunk);
    w.bwd = bwd_layout(batch, L, D, N).bytes;
    const size_t act = (size_t)(batch * L * D) * (dtype == SSM_BF16 ? 2 : 4);
    w.off_xc = w.bwd;
    w.off_gx = w.off_xc + round_up256(act);
    w.off_part = w.off_gx + round_up256(act);
    w.bytes = w.off_part + round_up256((size_t)(batch * w.nchunk * D * 5) * sizeof(float));
    return w;
}

size_t ssm_scan_bwd_conv_workspace_bytes(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype) {
    if (batch <= 0 || L <= 0 || D <= 0 || !supported_n(N)) return 0;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return 0;
    if (!bwd_sizes_ok(batch, L, D, N)) return 0;
    return conv_bwd_layout(batch, L, D, N, dtype).bytes;
}

int ssm_scan_bwd_conv(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                      const void *x_raw, const float *conv_w, const float *conv_b, const void *conv_state,
                      const void *delta_raw, const float *dt_bias, const float *A,
                      const void *Bt, const void *Ct, const float *Dskip, const void *z, const float *state_in,
                      const void *dy, const float *dstate,
                      void *dx_raw, float *dconv_w, float *dconv_b, void *dconv_state,
                      void *ddelta_raw, float *ddt_bias, float *dA, float *dBt, float *dCt,
                      float *dDskip, void *dz, float *dstate_in, void *workspace, size_t workspace_bytes,
                      void *stream) {
    if (batch < 0 || L < 0 || D < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!supported_n(N)) return SSM_ERR_UNSUPPORTED;
    if (!bwd_sizes_ok(batch, L, D, N)) return SSM_ERR_SHAPE;
    if (D > 0 && (!conv_w || !dconv_w)) return SSM_ERR_NULL;
    const void *ptrs[] = {conv_w, conv_b, conv_state, dconv_w, dconv_b, dconv_state};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    const bool tokens = batch > 0 && L > 0 && D > 0;
    if (tokens && (!x_raw || !dx_raw)) return SSM_ERR_NULL;
    if (x_raw && !aligned16(x_raw)) return SSM_ERR_ALIGN;
    if (dx_raw && !aligned16(dx_raw)) return SSM_ERR_ALIGN;
    const ConvBwdLayout w = tokens ? conv_bwd_layout(batch, L, D, N, dtype) : ConvBwdLayout{};
    if (tokens && (!workspace || workspace_bytes < w.bytes)) return SSM_ERR_WORKSPACE;
    if (workspace && !aligned16(workspace)) return SSM_ERR_ALIGN;
    char *ws = (char *)workspace;
    ssm::ConvBwdArgs c{};
    c.batch = batch;
    c.L = L;
    c.D = D;
    c.chunk = w.chunk;
    c.nchunk = w.nchunk;
    c.x_raw = x_raw;
    c.conv_state = conv_state;
    c.conv_w = conv_w;
    c.conv_b = conv_b;
    c.xc = tokens ? ws + w.off_xc : nullptr;
    c.gx = tokens ? ws + w.off_gx : nullptr;
    c.dx_raw = dx_raw;
    c.dconv_state = dconv_state;
    c.dconv_w = dconv_w;
    c.dconv_b = conv_b ? dconv_b : nullptr;
    c.part = tokens ? (float *)(ws + w.off_part) : nullptr;
    hipStream_t s = (hipStream_t)stream;
    // check the scan gradient's own arguments before launching anything: the
    // branch's output stands in for x (any aligned address passes the checks)
    const int chk = scan_bwd(batch, L, D, N, dtype, tokens ? c.xc : x_raw, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip,
                             z, state_in, dy, dstate, tokens ? ws + w.off_gx : dx_raw, ddelta_raw, ddt_bias, dA,
                             dBt, dCt, dDskip, dz, dstate_in, workspace, tokens ? w.bwd : workspace_bytes, stream,
                             TrapBwd{}, /*launch=*/false);
    if (chk != SSM_OK) return chk;
    if (D == 0) return SSM_OK;
    if (ssm::launch_conv_fwd(c, dtype, s) != hipSuccess) return SSM_ERR_HIP;
    const int rc = scan_bwd(batch, L, D, N, dtype, tokens ? c.xc : x_raw, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip,
                            z, state_in, dy, dstate, tokens ? ws + w.off_gx : dx_raw, ddelta_raw, ddt_bias, dA, dBt,
                            dCt, dDskip, dz, dstate_in, workspace, tokens ? w.bwd : workspace_bytes, stream);
    if (rc != SSM_OK) return rc;
    return ssm::launch_conv_bwd(c, dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_scan_bwd_dt(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype,
                    const void *x, const void *delta_raw, const float *dt_bias, const float *A,
                    const void *Bt, const void *Ct, const float *Dskip, const void *z, const float *state_in,
                    const void *dy, const float *dstate,
                    void *dx, void *ddelta_raw, float *ddt_bias, float *dA, float *dBt, float *dCt,
                    float *dDskip, void *dz, float *dstate_in, void *workspace, size_t workspace_bytes,
                    void *stream) {
    return scan_bwd(batch, L, D, N, dtype, x, delta_raw, dt_bias, 1, A, Bt, Ct, Dskip, z, state_in, dy, dstate,
                    dx, ddelta_raw, ddt_bias, dA, dBt, dCt, dDskip, dz, dstate_in, workspace, workspace_bytes,
                    stream);
}

int ssm_ssd_step(int64_t batch, int64_t H, int64_t P, int64_t G, int64_t N, int dtype,
                 const void *x, const void *delta, const float *A, const void *Bt, const void *Ct,
                 const float *Dskip, float *state, void *y, void *stream) {
    if (batch < 0 || H < 0 || P < 0 || G < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (!ssm::ssd_step_supported(P, N)) return SSM_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return SSM_ERR_SHAPE;
    if (checked_mul3(checked_mul(batch, H), P, N) < 0 || checked_mul3(batch, G, N) < 0 ||
        checked_mul(batch, H) >= ((int64_t)1 << 31))
        return SSM_ERR_SHAPE;
    if (batch == 0 || H == 0) return SSM_OK;
    if (!x || !delta || !A || !Bt || !Ct || !state || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bt, Ct, Dskip, state, y};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::SsdStepArgs a{};
    a.batch = batch;
    a.H = H;
    a.G = G;
    a.x = x;
    a.delta = delta;
    a.Bt = Bt;
    a.Ct = Ct;
    a.A = A;
    a.Dskip = Dskip;
    a.state = state;
    a.y = y;
    return ssm::launch_ssd_step(a, (int)N, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_ssd_fwd(int64_t batch, int64_t L, int64_t H, int64_t P, int64_t G, int64_t N, int dtype,
                const void *x, const void *delta, const float *A, const void *Bt, const void *Ct,
                const float *Dskip, const float *state_in, float *state_out, void *y, void *stream) {
    if (batch < 0 || L < 0 || H < 0 || P < 0 || G < 0 || N < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (dtype != SSM_BF16 || !ssm::ssd_supported(P, N)) return SSM_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return SSM_ERR_SHAPE;
    // 64 tokens of x and of Bt, Ct must span less than 4 GiB (32-bit offsets)
    if (H > ((int64_t)UINT32_MAX / (64 * 2 * 64)) || G * N > ((int64_t)UINT32_MAX / (2 * 64)))
        return SSM_ERR_UNSUPPORTED;
    if (checked_mul3(batch, L, H) < 0 || checked_mul3(checked_mul(batch, L), H, P) < 0 ||
        checked_mul3(checked_mul(batch, L), G, N) < 0 || checked_mul3(checked_mul(batch, H), P, N) < 0)
        return SSM_ERR_SHAPE;
    if (batch == 0 || H == 0) return SSM_OK;
    hipStream_t s = (hipStream_t)stream;
    if (L == 0) {
        if (!state_out) return SSM_OK;
        if (!aligned16(state_out) || (state_in && !aligned16(state_in))) return SSM_ERR_ALIGN;
        if (state_in == state_out) return SSM_OK;
        return ssm::launch_state_copy(state_in, state_out, batch * H * P * N, s) == hipSuccess ? SSM_OK
                                                                                              : SSM_ERR_HIP;
    }
    if (!x || !delta || !A || !Bt || !Ct || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bt, Ct, Dskip, state_in, state_out, y};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::SsdArgs a{};
    a.batch = batch;
    a.L = L;
    a.H = H;
    a.G = G;
    a.x = x;
    a.delta = delta;
    a.Bt = Bt;
    a.Ct = Ct;
    a.A = A;
    a.Dskip = Dskip;
    a.state_in = state_in;
    a.state_out = state_out;
    a.y = y;
    return ssm::launch_ssd(a, (int)N, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

// Sizes and arguments that ssm_ssd_fwd_cache and ssm_ssd_step_cache share;
// fills `a` when everything is in order.
static int ssd_cache_check(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N, int dtype,
                           bool prompt, const int32_t *cu_seqlens, const int32_t *slots, const int32_t *resume,
                           int64_t num_slots, const void *xBC, int64_t xBC_stride, const float *conv_w,
                           const float *conv_b, const void *dt_raw, int64_t dt_stride, const float *dt_bias,
                           const float *A, const float *Dskip, void *conv_cache, float *state_cache, void *y,
                           const void *workspace, size_t workspace_bytes, ssm::SsdCacheArgs *a) {
    if (seqs < 0 || rows < 0 || H < 0 || P < 0 || G < 0 || N < 0 || num_slots < 0 || xBC_stride < 0 || dt_stride < 0)
        return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if ((prompt && dtype != SSM_BF16) || !ssd_cache_sizes(seqs, rows, H, P, G, N)) return SSM_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return SSM_ERR_SHAPE;
    const int64_t C = H * P + 2 * G * N;
    if (num_slots > INT32_MAX || xBC_stride < C || dt_stride < H) return SSM_ERR_SHAPE;
    // 64 rows and the three before them are reached by 32-bit offsets
    if (xBC_stride >= kMaxRow || dt_stride >= kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (checked_mul3(checked_mul(num_slots, H), P, N) < 0 || checked_mul3(num_slots, C, 3) < 0) return SSM_ERR_SHAPE;
    if (seqs == 0 || H == 0) return SSM_OK;
    if (!slots || !A || !conv_w || !conv_cache || !state_cache || (prompt && !cu_seqlens)) return SSM_ERR_NULL;
    if (rows > 0 && (!xBC || !dt_raw || !y)) return SSM_ERR_NULL;
    const void *ptrs[] = {cu_seqlens, slots, resume, xBC, conv_w, conv_b, dt_raw, dt_bias, A, Dskip,
                          conv_cache, state_cache, y, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    if (xBC_stride * (dtype == SSM_F32 ? 4 : 2) % 16 != 0) return SSM_ERR_ALIGN;
    const size_t need = prompt ? ssm_ssd_fwd_cache_workspace_bytes(seqs, rows, H, P, G, N, dtype)
                               : ssm_ssd_step_cache_workspace_bytes(seqs, H, P, G, N);
    if (!workspace || workspace_bytes < need) return SSM_ERR_WORKSPACE;
    a->seqs = seqs;
    a->rows = rows;
    a->H = H;
    a->P = P;
    a->G = G;
    a->C = C;
    a->num_slots = num_slots;
    a->xBC_stride = xBC_stride;
    a->dt_stride = dt_stride;
    a->cu_seqlens = cu_seqlens;
    a->slots = slots;
    a->resume = resume;
    a->xBC = xBC;
    a->dt_raw = dt_raw;
    a->conv_w = conv_w;
    a->conv_b = conv_b;
    a->dt_bias = dt_bias;
    a->A = A;
    a->Dskip = Dskip;
    a->conv_cache = conv_cache;
    a->state_cache = state_cache;
    a->y = y;
    return SSM_OK;
}

size_t ssm_ssd_fwd_cache_workspace_bytes(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N,
                                         int dtype) {
    if (dtype != SSM_BF16 || seqs <= 0 || rows < 0 || H <= 0 || G < 1 || H % G != 0 ||
        !ssd_cache_sizes(seqs, rows, H, P, G, N))
        return 0;
    return ssm::ssd_cache_workspace(seqs, rows, H, P, G, N);
}

int ssm_ssd_fwd_cache(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N, int dtype,
                      const int32_t *cu_seqlens, const int32_t *slots, const int32_t *resume, int64_t num_slots,
                      const void *xBC, int64_t xBC_stride, const float *conv_w, const float *conv_b,
                      const void *dt_raw, int64_t dt_stride, const float *dt_bias, const float *A,
                      const float *Dskip, void *conv_cache, float *state_cache, void *y, void *workspace,
                      size_t workspace_bytes, void *stream) {
    ssm::SsdCacheArgs a{};
    const int st = ssd_cache_check(seqs, rows, H, P, G, N, dtype, true, cu_seqlens, slots, resume, num_slots, xBC,
                                   xBC_stride, conv_w, conv_b, dt_raw, dt_stride, dt_bias, A, Dskip, conv_cache,
                                   state_cache, y, workspace, workspace_bytes, &a);
    if (st != SSM_OK || seqs == 0 || H == 0) return st;
    return ssm::launch_ssd_cache(a, (int)N, workspace, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_ssd_step_cache_workspace_bytes(int64_t batch, int64_t H, int64_t P, int64_t G, int64_t N) {
    if (batch <= 0 || H <= 0 || G < 1 || H % G != 0 || !ssd_cache_sizes(batch, batch, H, P, G, N)) return 0;
    return round_up256((size_t)batch * 4) + (size_t)batch * ssd_step_row(H, P, G, N) * 4;
}

int ssm_ssd_step_cache(int64_t batch, int64_t H, int64_t P, int64_t G, int64_t N, int dtype, const int32_t *slots,
                       int64_t num_slots, const void *xBC, int64_t xBC_stride, const float *conv_w,
                       const float *conv_b, const void *dt_raw, int64_t dt_stride, const float *dt_bias,
                       const float *A, const float *Dskip, void *conv_cache, float *state_cache, void *y,
                       void *workspace, size_t workspace_bytes, void *stream) {
    ssm::SsdCacheArgs a{};
    const int st = ssd_cache_check(batch, batch, H, P, G, N, dtype, false, nullptr, slots, nullptr, num_slots, xBC,
                                   xBC_stride, conv_w, conv_b, dt_raw, dt_stride, dt_bias, A, Dskip, conv_cache,
                                   state_cache, y, workspace, workspace_bytes, &a);
    if (st != SSM_OK || batch == 0 || H == 0) return st;
    a.ws_slot = (int32_t *)workspace;
    a.ws_act = (float *)((char *)workspace + round_up256((size_t)batch * 4));
    a.ws_row = ssd_step_row(H, P, G, N);
    return ssm::launch_ssd_step_cache(a, (int)N, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0 || checked_mul(rows, D) < 0) return 0;
    return (size_t)ssm::norm_bwd_blocks(rows) * 2 * (size_t)D * sizeof(float);
}

// Sizes that every norm entry point takes.
static int norm_check(int64_t rows, int64_t D, int64_t groups, int dtype) {
    if (rows < 0 || D < 0 || groups < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if (D > 0 && (groups < 1 || D % groups != 0)) return SSM_ERR_SHAPE;
    if (D > 0 && (D / groups > ssm::kNormMaxWidth || groups > 65535 || D > kMaxNorm)) return SSM_ERR_UNSUPPORTED;
    return checked_mul(rows, D) < 0 ? SSM_ERR_SHAPE : SSM_OK;
}

int ssm_add_norm_fwd(int64_t rows, int64_t D, int dtype, int res_dtype, const void *x, const void *residual,
                     const float *scale, const float *weight, float eps, void *y, void *residual_out, void *stream) {
    const int st = norm_check(rows, D, 1, dtype);
    if (st != SSM_OK) return st;
    if (res_dtype != SSM_F32 && res_dtype != dtype) return SSM_ERR_DTYPE;
    if (rows == 0 || D == 0) return SSM_OK;
    if (!x || !weight || !y || !residual_out) return SSM_ERR_NULL;
    const void *ptrs[] = {x, residual, scale, weight, y, residual_out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::AddNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    a.x = x;
    a.residual = residual;
    a.scale = scale;
    a.weight = weight;
    a.y = y;
    a.residual_out = residual_out;
    return ssm::launch_add_norm(a, false, dtype, res_dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_add_norm_bwd(int64_t rows, int64_t D, int dtype, int res_dtype, const void *dy, const void *r,
                     const float *weight, const void *x, const float *scale, const void *dres, float eps, void *dx,
                     void *dresidual, float *dweight, float *dscale, void *workspace, size_t workspace_bytes,
                     void *stream) {
    const int st = norm_check(rows, D, 1, dtype);
    if (st != SSM_OK) return st;
    if (res_dtype != SSM_F32 && res_dtype != dtype) return SSM_ERR_DTYPE;
    if (D == 0) return SSM_OK;
    if (!dweight) return SSM_ERR_NULL;
    if (rows > 0 && (!dy || !r || !weight || !dx || !dresidual || (scale && !x))) return SSM_ERR_NULL;
    const void *ptrs[] = {dy, r, weight, x, scale, dres, dx, dresidual, dweight, dscale, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    if (rows == 0) {
        if (ssm::launch_state_copy(nullptr, dweight, D, s) != hipSuccess) return SSM_ERR_HIP;
        return !dscale || ssm::launch_state_copy(nullptr, dscale, D, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    }
    if (!workspace || workspace_bytes < ssm_norm_bwd_workspace_bytes(rows, D)) return SSM_ERR_WORKSPACE;
    ssm::AddNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    a.x = x;
    a.residual = r;
    a.dy = dy;
    a.dres = dres;
    a.scale = scale;
    a.weight = weight;
    a.residual_out = dresidual;
    a.dx = dx;
    a.dweight = dweight;
    a.dscale = scale ? dscale : nullptr;
    a.part = (float *)workspace;
    return ssm::launch_add_norm(a, true, dtype, res_dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_gate_norm_fwd(int64_t rows, int64_t D, int64_t groups, int dtype, const void *x, int64_t x_stride,
                      const void *z, int64_t z_stride, const float *weight, float eps, void *y, void *stream) {
    const int st = norm_check(rows, D, groups, dtype);
    if (st != SSM_OK) return st;
    if (x_stride < D || z_stride < D || checked_mul(rows, x_stride) < 0 || checked_mul(rows, z_stride) < 0)
        return SSM_ERR_SHAPE;
    if (rows == 0 || D == 0) return SSM_OK;
    if (!x || !z || !weight || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, z, weight, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return SSM_ERR_ALIGN;
    ssm::GateNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.groups = groups;
    a.x_stride = x_stride;
    a.z_stride = z_stride;
    a.eps = eps;
    a.x = x;
    a.z = z;
    a.weight = weight;
    a.y = y;
    return ssm::launch_gate_norm(a, false, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_gate_norm_bwd(int64_t rows, int64_t D, int64_t groups, int dtype, const void *dy, const void *x,
                      int64_t x_stride, const void *z, int64_t z_stride, const float *weight, float eps, void *dx,
                      void *dz, int64_t dz_stride, float *dweight, void *workspace, size_t workspace_bytes,
                      void *stream) {
    const int st = norm_check(rows, D, groups, dtype);
    if (st != SSM_OK) return st;
    if (x_stride < D || z_stride < D || dz_stride < D || checked_mul(rows, x_stride) < 0 ||
        checked_mul(rows, z_stride) < 0 || checked_mul(rows, dz_stride) < 0)
        return SSM_ERR_SHAPE;
    if (D == 0) return SSM_OK;
    if (!dweight) return SSM_ERR_NULL;
    if (rows > 0 && (!dy || !x || !z || !weight || !dx || !dz)) return SSM_ERR_NULL;
    const void *ptrs[] = {dy, x, z, weight, dx, dz, dweight, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    if (rows == 0)
        return ssm::launch_state_copy(nullptr, dweight, D, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
    if (!workspace || workspace_bytes < ssm_norm_bwd_workspace_bytes(rows, D)) return SSM_ERR_WORKSPACE;
    ssm::GateNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.groups = groups;
    a.x_stride = x_stride;
    a.z_stride = z_stride;
    a.dz_stride = dz_stride;
    a.eps = eps;
    a.x = x;
    a.z = z;
    a.dy = dy;
    a.weight = weight;
    a.dx = dx;
    a.dz = dz;
    a.dweight = dweight;
    a.part = (float *)workspace;
    return ssm::launch_gate_norm(a, true, dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

// Sizes that the gated delta rule takes: threads of a launch per chunk of 64 tokens
// (or request) and 64 rows of a head's state; of the prompts' walk, four per row, the
// groups of all sequences rounded up to whole eights.
static bool delta_sizes(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N, bool prompt) {
    if (P < 64 || P > 256 || P % 64 != 0 || (N != 64 && N != 128)) return false;
    if (seqs > 65535 || rows > INT32_MAX || H > 65535 || H >= kMaxRow / P || G >= kMaxRow / N) return false;
    if (prompt && G > 0 && (G * seqs + 7) / 8 * 8 * (H / G) * P * 4 > UINT32_MAX) return false;
    return (rows / 64 + seqs) * (H * P / 64 * 256 + G * 512) <= UINT32_MAX;
}

static int delta_check(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N, int dtype, bool prompt,
                       const int32_t *cu_seqlens, const int32_t *slots, const int32_t *resume, int64_t num_slots,
                       const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                       int64_t v_stride, const void *dt_raw, int64_t dt_stride, const float *dt_bias,
                       const void *beta_raw, int64_t beta_stride, const float *A, float scale, float norm_eps,
                       float *state_cache, void *y, ssm::DeltaArgs *a) {
    if (seqs < 0 || rows < 0 || H < 0 || P < 0 || G < 0 || N < 0 || num_slots < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    if ((prompt && dtype != SSM_BF16) || !delta_sizes(seqs, rows, H, P, G, N, prompt)) return SSM_ERR_UNSUPPORTED;
    if (H > 0 && (G < 1 || H % G != 0)) return SSM_ERR_SHAPE;
    if (num_slots > INT32_MAX || q_stride < G * N || k_stride < G * N || v_stride < H * P || dt_stride < H ||
        beta_stride < H)
        return SSM_ERR_SHAPE;
    const int64_t strides[] = {q_stride, k_stride, v_stride, dt_stride, beta_stride};
    for (const int64_t n : strides)
        if (n >= kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (checked_mul3(checked_mul(num_slots, H), P, N) < 0) return SSM_ERR_SHAPE;
    if (seqs == 0 || H == 0) return SSM_OK;
    if (!slots || !A || !state_cache || (prompt && !cu_seqlens)) return SSM_ERR_NULL;
    if (rows > 0 && (!q || !k || !v || !dt_raw || !beta_raw || !y)) return SSM_ERR_NULL;
    const void *ptrs[] = {cu_seqlens, slots, resume, q, k, v, dt_bias, A, state_cache, y};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    const int64_t size = dtype == SSM_F32 ? 4 : 2;
    if ((uintptr_t)dt_raw % size != 0 || (uintptr_t)beta_raw % size != 0 || q_stride * size % 16 != 0 ||
        k_stride * size % 16 != 0 || v_stride * size % 16 != 0)
        return SSM_ERR_ALIGN;
    a->seqs = seqs;
    a->rows = rows;
    a->H = H;
    a->P = P;
    a->G = G;
    a->num_slots = num_slots;
    a->q_stride = q_stride;
    a->k_stride = k_stride;
    a->v_stride = v_stride;
    a->dt_stride = dt_stride;
    a->beta_stride = beta_stride;
    a->cu_seqlens = cu_seqlens;
    a->slots = slots;
    a->resume = resume;
    a->q = q;
    a->k = k;
    a->v = v;
    a->dt_raw = dt_raw;
    a->beta_raw = beta_raw;
    a->dt_bias = dt_bias;
    a->A = A;
    a->scale = scale;
    a->norm_eps = norm_eps;
    a->state_cache = state_cache;
    a->y = y;
    return SSM_OK;
}

size_t ssm_delta_fwd_cache_workspace_bytes(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N,
                                           int dtype) {
    if (dtype != SSM_BF16 || seqs <= 0 || rows < 0 || H <= 0 || G < 1 || H % G != 0 ||
        !delta_sizes(seqs, rows, H, P, G, N, true))
        return 0;
    return ssm::delta_workspace(seqs, rows, H, P, G, N);
}

int ssm_delta_fwd_cache(int64_t seqs, int64_t rows, int64_t H, int64_t P, int64_t G, int64_t N, int dtype,
                        const int32_t *cu_seqlens, const int32_t *slots, const int32_t *resume, int64_t num_slots,
                        const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                        int64_t v_stride, const void *dt_raw, int64_t dt_stride, const float *dt_bias,
                        const void *beta_raw, int64_t beta_stride, const float *A, float scale, float norm_eps,
                        float *state_cache, void *y, void *workspace, size_t workspace_bytes, void *stream) {
    ssm::DeltaArgs a{};
    const int st = delta_check(seqs, rows, H, P, G, N, dtype, true, cu_seqlens, slots, resume, num_slots, q, q_stride,
                               k, k_stride, v, v_stride, dt_raw, dt_stride, dt_bias, beta_raw, beta_stride, A, scale,
                               norm_eps, state_cache, y, &a);
    if (st != SSM_OK || seqs == 0 || H == 0) return st;
    if (workspace && !aligned16(workspace)) return SSM_ERR_ALIGN;
    if (!workspace || workspace_bytes < ssm::delta_workspace(seqs, rows, H, P, G, N)) return SSM_ERR_WORKSPACE;
    return ssm::launch_delta(a, (int)N, workspace, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_delta_step_cache(int64_t batch, int64_t H, int64_t P, int64_t G, int64_t N, int dtype, const int32_t *slots,
                         int64_t num_slots, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                         const void *v, int64_t v_stride, const void *dt_raw, int64_t dt_stride,
                         const float *dt_bias, const void *beta_raw, int64_t beta_stride, const float *A, float scale,
                         float norm_eps, float *state_cache, void *y, void *stream) {
    ssm::DeltaArgs a{};
    const int st = delta_check(batch, batch, H, P, G, N, dtype, false, nullptr, slots, nullptr, num_slots, q, q_stride,
                               k, k_stride, v, v_stride, dt_raw, dt_stride, dt_bias, beta_raw, beta_stride, A, scale,
                               norm_eps, state_cache, y, &a);
    if (st != SSM_OK || batch == 0 || H == 0) return st;
    return ssm::launch_delta_step(a, (int)N, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

static int conv_cache(int64_t seqs, int64_t rows, int64_t C, int dtype, bool prompt, const int32_t *cu_seqlens,
                      const int32_t *slots, const int32_t *resume, int64_t num_slots, const void *x, int64_t x_stride,
                      const float *conv_w, const float *conv_b, void *conv_cache, void *y, void *stream) {
    if (seqs < 0 || rows < 0 || C < 0 || num_slots < 0) return SSM_ERR_SHAPE;
    if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_DTYPE;
    // threads of a launch: 256 per 64 tokens (or request) and, at the least, 256 channels
    if (seqs > 65535 || rows > INT32_MAX || C >= kMaxRow ||
        ((prompt ? rows / 64 : 0) + seqs) * ((C + 255) / 256) * 256 > UINT32_MAX)
        return SSM_ERR_UNSUPPORTED;
    if (num_slots > INT32_MAX || x_stride < C || checked_mul3(num_slots, C, 3) < 0) return SSM_ERR_SHAPE;
    if (x_stride >= kMaxRow) return SSM_ERR_UNSUPPORTED;
    if (seqs == 0 || C == 0) return SSM_OK;
    if (!slots || !conv_w || !conv_cache || (prompt && !cu_seqlens) || (rows > 0 && (!x || !y))) return SSM_ERR_NULL;
    const void *ptrs[] = {cu_seqlens, slots, resume, x, conv_w, conv_b, conv_cache, y};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::ConvCacheArgs a{};
    a.seqs = seqs;
    a.rows = rows;
    a.C = C;
    a.num_slots = num_slots;
    a.x_stride = x_stride;
    a.cu_seqlens = cu_seqlens;
    a.slots = slots;
    a.resume = resume;
    a.x = x;
    a.conv_w = conv_w;
    a.conv_b = conv_b;
    a.conv_cache = conv_cache;
    a.y = y;
    return ssm::launch_conv_cache(a, prompt, dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_conv_fwd_cache(int64_t seqs, int64_t rows, int64_t C, int dtype, const int32_t *cu_seqlens,
                       const int32_t *slots, const int32_t *resume, int64_t num_slots, const void *x,
                       int64_t x_stride, const float *conv_w, const float *conv_b, void *cache, void *y,
                       void *stream) {
    return conv_cache(seqs, rows, C, dtype, true, cu_seqlens, slots, resume, num_slots, x, x_stride, conv_w, conv_b,
                      cache, y, stream);
}

int ssm_conv_step_cache(int64_t batch, int64_t C, int dtype, const int32_t *slots, int64_t num_slots, const void *x,
                        int64_t x_stride, const float *conv_w, const float *conv_b, void *cache, void *y,
                        void *stream) {
    return conv_cache(batch, batch, C, dtype, false, nullptr, slots, nullptr, num_slots, x, x_stride, conv_w, conv_b,
                      cache, y, stream);
}

int ssm_add_layer_norm_fwd(int64_t rows, int64_t D, int dtype, int res_dtype, const void *x, const void *residual,
                           const float *scale, const float *weight, const float *bias, float eps, void *y,
                           void *residual_out, void *stream) {
    const int st = norm_check(rows, D, 1, dtype);
    if (st != SSM_OK) return st;
    if (res_dtype != SSM_F32 && res_dtype != dtype) return SSM_ERR_DTYPE;
    if (rows == 0 || D == 0) return SSM_OK;
    if (!x || !weight || !y) return SSM_ERR_NULL;
    const void *ptrs[] = {x, residual, scale, weight, bias, y, residual_out};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    ssm::LayerNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    a.x = x;
    a.residual = residual;
    a.scale = scale;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.residual_out = residual_out;
    return ssm::launch_layer_norm(a, false, dtype, res_dtype, (hipStream_t)stream) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

size_t ssm_add_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0 || checked_mul(rows, D) < 0) return 0;
    return (size_t)ssm::norm_bwd_blocks(rows) * 3 * (size_t)D * sizeof(float);
}

int ssm_add_layer_norm_bwd(int64_t rows, int64_t D, int dtype, int res_dtype, const void *dy, const void *r,
                           const float *weight, const void *x, const float *scale, const void *dres, float eps,
                           void *dx, void *dresidual, float *dweight, float *dbias, float *dscale, void *workspace,
                           size_t workspace_bytes, void *stream) {
    const int st = norm_check(rows, D, 1, dtype);
    if (st != SSM_OK) return st;
    if (res_dtype != SSM_F32 && res_dtype != dtype) return SSM_ERR_DTYPE;
    if (D == 0) return SSM_OK;
    if (!dweight || !dbias) return SSM_ERR_NULL;
    if (rows > 0 && (!dy || !r || !weight || !dx || (scale && !x))) return SSM_ERR_NULL;
    const void *ptrs[] = {dy, r, weight, x, scale, dres, dx, dresidual, dweight, dbias, dscale, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return SSM_ERR_ALIGN;
    hipStream_t s = (hipStream_t)stream;
    if (rows == 0) {
        float *sums[] = {dweight, dbias, dscale};
        for (float *p : sums)
            if (p && ssm::launch_state_copy(nullptr, p, D, s) != hipSuccess) return SSM_ERR_HIP;
        return SSM_OK;
    }
    if (!workspace || workspace_bytes < ssm_add_layer_norm_bwd_workspace_bytes(rows, D)) return SSM_ERR_WORKSPACE;
    ssm::LayerNormArgs a{};
    a.rows = rows;
    a.D = D;
    a.eps = eps;
    a.x = x;
    a.residual = r;
    a.dy = dy;
    a.dres = dres;
    a.scale = scale;
    a.weight = weight;
    a.residual_out = dresidual;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dscale = scale ? dscale : nullptr;
    a.part = (float *)workspace;
    return ssm::launch_layer_norm(a, true, dtype, res_dtype, s) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"

namespace ssm {

int scan_fwd_euler(int64_t batch, int64_t L, int64_t D, int64_t N, int dtype, const void *x, const void *delta,
                   const float *A, const void *Bt, const void *Ct, const float *Dskip, const void *z,
                   const float *state_in, float *state_out, void *y, void *workspace, size_t workspace_bytes,
                   void *stream, bool launch) {
    return scan_fwd(batch, L, D, N, dtype, x, delta, nullptr, 0, A, Bt, Ct, Dskip, z, state_in, state_out, y,
                    workspace, workspace_bytes, stream, TrapIn{}, launch);
}

}  // namespace ssm
