// C ABI of the stand-alone operators: grouped products and their gradients,
// 4-bit matrix-vector products, block norms.  Argument validation, workspace
// layout and launches; contracts in include/moe.h.  Nothing here allocates,
// synchronises or copies to the host.
#include <math.h>
#include <string.h>

#include "moe.h"
#include "moe_ops.h"

namespace moe {
void set_last_error(const char* text);
}

namespace {

static_assert((int)moe::DT_BF16 == (int)MOE_DT_BF16 && (int)moe::DT_F16 == (int)MOE_DT_F16 &&
                  (int)moe::DT_F32 == (int)MOE_DT_F32,
              "type codes");

size_t align_up(size_t v) { return (v + 255) / 256 * 256; }

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A pointer that must be there, and its alignment.
int need(const void* p, size_t a)
{
    if (!p) return MOE_ERR_INVALID_ARG;
    return aligned(p, a) ? MOE_OK : MOE_ERR_MISALIGNED;
}
// One that may be null.
int maybe(const void* p, size_t a) { return aligned(p, a) ? MOE_OK : MOE_ERR_MISALIGNED; }

int hip_status(hipError_t e)
{
    if (e == hipSuccess) return MOE_OK;
    moe::set_last_error(hipGetErrorString(e));
    return MOE_ERR_HIP;
}

size_t type_bytes(int dtype) { return dtype == MOE_DT_F32 ? 4 : 2; }

constexpr int kMaxExperts = 256, kMaxTopK = 8, kMaxWidth = 1 << 22;

// Sizes shared by the products over sorted rows.
int check_rows(int M, int N, int K, int E, int T, int k)
{
    if (M < 0 || N <= 0 || K <= 0 || E <= 0 || T < 0 || k < 1) return MOE_ERR_INVALID_ARG;
    if (E > kMaxExperts || k > kMaxTopK || N > kMaxWidth || K > kMaxWidth) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)E * N * K > (int64_t)1 << 37) return MOE_ERR_UNSUPPORTED;
    // A launch holds fewer than 2^32 threads, 256 in a workgroup; tiles of 128 x 64.
    const int64_t most = ((int64_t)1 << 24) - 16, wide = (N > K ? N : K) / 64 + 1;
    if (wide * ((int64_t)M / 64 + E + 1) > most) return MOE_ERR_UNSUPPORTED;
    if (((int64_t)N / 64 + 1) * ((int64_t)K / 128 + 2) * E > most) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// The rows' segments: expert_offsets may be null for one expert; with
// sorted_pairs the rows come from T rows, k pairs each.
int check_segments(int E, int T, const int32_t* offsets, const int32_t* pairs)
{
    if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (pairs && T < 1) return MOE_ERR_INVALID_ARG;
    int rc;
    if ((rc = maybe(offsets, 4)) || (rc = maybe(pairs, 4))) return rc;
    return MOE_OK;
}

int check_gmm(const moe_gmm* g)
{
    if (!g) return MOE_ERR_INVALID_ARG;
    int rc = check_rows(g->M, g->N, g->K, g->E, g->T, g->k);
    if (rc) return rc;
    if (g->dtype != MOE_DT_BF16 && g->dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
    if (g->out_dtype != g->dtype && g->out_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (g->accumulate != 0 && g->accumulate != 1) return MOE_ERR_INVALID_ARG;
    if ((g->lda != 0 && g->lda < g->K) || (g->ldc != 0 && g->ldc < g->N)) return MOE_ERR_INVALID_ARG;
    if (g->lda > (int64_t)1 << 31 || g->ldc > (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe::GmmArgs gmm_args(const moe_gmm& g, const int32_t* offsets, const int32_t* pairs)
{
    moe::GmmArgs a;
    memset(&a, 0, sizeof a);
    a.M = g.M;
    a.N = g.N;
    a.K = g.K;
    a.E = g.E;
    a.a_rows = pairs ? g.T : g.M;
    a.k = g.k;
    a.dtype = g.dtype;
    a.out_dtype = g.out_dtype;
    a.accumulate = g.accumulate;
    a.lda = g.lda ? g.lda : g.K;
    a.ldc = g.ldc ? g.ldc : g.N;
    a.offsets = offsets;
    a.pairs = pairs;
    return a;
}

struct WgradLayout {
    size_t part, dbias, total;
};
WgradLayout wgrad_layout(const moe_gmm& g)
{
    WgradLayout L;
    const int sp = moe::gmm_wgrad_splits(g.M, g.N, g.K, g.E);
    L.part = 0;
    L.dbias = align_up(sp > 1 ? (size_t)sp * g.E * g.N * g.K * 4 : 0);
    L.total = L.dbias + align_up((size_t)moe::gmm_dbias_ranges(g.M, g.E) * g.N * 4);
    return L;
}

int check_w4(const moe_w4* d)
{
    if (!d) return MOE_ERR_INVALID_ARG;
    int rc = check_rows(d->M, d->N, d->K, d->E, d->T, d->k);
    if (rc) return rc;
    if (d->K % 32 != 0) return MOE_ERR_UNSUPPORTED;
    if (d->group != 32 && d->group != 64 && d->group != 128) return MOE_ERR_UNSUPPORTED;
    if (d->dtype != MOE_DT_BF16 && d->dtype != MOE_DT_F16) return MOE_ERR_UNSUPPORTED;
    if (d->out_dtype != d->dtype && d->out_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (d->act != MOE_ACT_NONE && d->act != MOE_ACT_SWIGLU) return MOE_ERR_UNSUPPORTED;
    if (d->act == MOE_ACT_SWIGLU && d->N % 2 != 0) return MOE_ERR_INVALID_ARG;
    // work items are counted in 32 bits, whatever the offsets say
    const int64_t passes = d->M <= 4 * d->E ? d->M / 4 + 1 : d->M / 16 + 1;
    if (passes * d->E * ((int64_t)d->N / 32 + 1) > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int check_norm(const moe_norm* d)
{
    if (!d || d->T < 0 || d->H <= 0) return MOE_ERR_INVALID_ARG;
    if (d->H > moe::NORM_MAX_H) return MOE_ERR_UNSUPPORTED;
    if (d->dtype < MOE_DT_BF16 || d->dtype > MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (d->wdtype != d->dtype && d->wdtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if (d->kind < MOE_NORM_NONE || d->kind > MOE_NORM_LAYER) return MOE_ERR_UNSUPPORTED;
    if (d->gate < MOE_GATE_NONE || d->gate > MOE_GATE_FULL) return MOE_ERR_UNSUPPORTED;
    if (!(d->eps >= 0.f) || isinf(d->eps) || !isfinite(d->res_scale)) return MOE_ERR_INVALID_ARG;
    if (!(d->dropout_p >= 0.f) || d->dropout_p >= 1.f || lrintf(d->dropout_p * 65536.f) > 65535)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe::NormArgs norm_args(const moe_norm& d, bool out)
{
    moe::NormArgs a;
    memset(&a, 0, sizeof a);
    a.T = d.T;
    a.H = d.H;
    a.dtype = d.dtype;
    a.wdtype = d.wdtype;
    a.kind = d.kind;
    a.gate_kind = out ? d.gate : 0;
    a.eps = d.eps;
    a.res_scale = d.res_scale;
    a.drop_threshold = out ? (uint32_t)lrintf(d.dropout_p * 65536.f) : 0;
    a.drop_scale = 65536.f / (float)(65536 - (int)a.drop_threshold);
    return a;
}

// The parameters of a norm and, after the block, of its gate and dropout.
int check_norm_params(const moe_norm& d, bool out, const void* weight, const void* bias, const void* gate,
                      const uint64_t* rng)
{
    const size_t wb = type_bytes(d.wdtype);
    int rc;
    if (d.kind == MOE_NORM_NONE && (weight || bias || !out)) return MOE_ERR_INVALID_ARG;
    if ((rc = maybe(weight, wb)) || (rc = maybe(bias, wb))) return rc;
    if (!out) return MOE_OK;
    if ((d.gate != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
    if ((rc = maybe(gate, type_bytes(d.dtype)))) return rc;
    if (lrintf(d.dropout_p * 65536.f) > 0 && (rc = need(rng, 8))) return rc;
    return MOE_OK;
}

size_t norm_ws_bytes(const moe_norm& d) { return align_up(moe::norm_partial_floats(d.T, d.H) * sizeof(float)); }

int check_norm_ws(const moe_norm& d, const void* ws, size_t bytes)
{
    if (bytes < norm_ws_bytes(d)) return MOE_ERR_WORKSPACE;
    return need(ws, 16);
}

}  // namespace

extern "C" {

int moe_grouped_mm(const moe_gmm* g, const void* a, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                   const void* b, const void* bias, void* c, void* stream)
{
    int rc = check_gmm(g);
    if (rc) return rc;
    if (g->accumulate) return MOE_ERR_UNSUPPORTED;
    if (g->M == 0) return MOE_OK;
    if ((rc = check_segments(g->E, g->T, expert_offsets, sorted_pairs)) || (rc = need(a, 2)) || (rc = need(b, 2)) ||
        (rc = maybe(bias, 2)) || (rc = need(c, type_bytes(g->out_dtype))))
        return rc;
    moe::GmmArgs x = gmm_args(*g, expert_offsets, sorted_pairs);
    x.a = a;
    x.b = b;
    x.bias = bias;
    x.out = c;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(moe::gmm_use_skinny(x) ? moe::launch_gmm_skinny(x, s) : moe::launch_gmm_forward(x, s));
}

int moe_grouped_mm_dgrad(const moe_gmm* g, const void* dc, const int32_t* expert_offsets, const void* b, void* da,
                         void* stream)
{
    int rc = check_gmm(g);
    if (rc) return rc;
    if (g->accumulate) return MOE_ERR_UNSUPPORTED;
    if (g->M == 0) return MOE_OK;
    if ((rc = check_segments(g->E, g->T, expert_offsets, nullptr)) || (rc = need(dc, 2)) || (rc = need(b, 2)) ||
        (rc = need(da, type_bytes(g->out_dtype))))
        return rc;
    moe::GmmArgs x = gmm_args(*g, expert_offsets, nullptr);
    x.dc = dc;
    x.b = b;
    x.out = da;
    return hip_status(moe::launch_gmm_dgrad(x, static_cast<hipStream_t>(stream)));
}

int moe_grouped_mm_workspace_size(const moe_gmm* g, size_t* bytes)
{
    int rc = check_gmm(g);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = wgrad_layout(*g).total;
    return MOE_OK;
}

int moe_grouped_mm_wgrad(const moe_gmm* g, const void* a, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                         const void* dc, void* db, float* dbias, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_gmm(g);
    if (rc) return rc;
    if (g->accumulate && g->out_dtype != MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
    if ((rc = need(db, type_bytes(g->out_dtype))) || (rc = maybe(dbias, 4))) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (g->M == 0) {  // no rows: the gradients are zero, or what was accumulated so far
        if (g->accumulate) return MOE_OK;
        const int64_t n = (int64_t)g->E * g->N * g->K * (type_bytes(g->out_dtype) / 2);
        if ((rc = hip_status(moe::launch_zero16(db, n, s)))) return rc;
        return hip_status(moe::launch_zero16(dbias, (int64_t)g->E * g->N * 2, s));
    }
    if ((rc = check_segments(g->E, g->T, expert_offsets, sorted_pairs)) || (rc = need(a, 2)) || (rc = need(dc, 2)))
        return rc;
    const WgradLayout L = wgrad_layout(*g);
    if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
    if ((rc = need(workspace, 16))) return rc;
    moe::GmmArgs x = gmm_args(*g, expert_offsets, sorted_pairs);
    x.a = a;
    x.dc = dc;
    x.out = db;
    x.dbias = dbias;
    x.splits = moe::gmm_wgrad_splits(g->M, g->N, g->K, g->E);
    x.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.part);
    x.dbias_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.dbias);
    return hip_status(moe::launch_gmm_wgrad(x, s));
}

int moe_w4_matvec(const moe_w4* d, const void* x, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                  const uint8_t* codes, const void* scales, const uint8_t* zeros, const void* bias, void* y,
                  void* stream)
{
    int rc = check_w4(d);
    if (rc) return rc;
    if (d->M == 0) return MOE_OK;
    if ((rc = check_segments(d->E, d->T, expert_offsets, sorted_pairs)) || (rc = need(x, 16)) ||
        (rc = need(codes, 16)) || (rc = need(scales, 2)) || (rc = maybe(bias, 2)) ||
        (rc = need(y, type_bytes(d->out_dtype))))
        return rc;
    moe::W4Args a;
    memset(&a, 0, sizeof a);
    a.M = d->M;
    a.N = d->N;
    a.K = d->K;
    a.E = d->E;
    a.x_rows = sorted_pairs ? d->T : d->M;
    a.k = d->k;
    a.group = d->group;
    a.dtype = d->dtype;
    a.out_dtype = d->out_dtype;
    a.swiglu = d->act == MOE_ACT_SWIGLU;
    a.offsets = expert_offsets;
    a.pairs = sorted_pairs;
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    a.zeros = zeros;
    a.bias = bias;
    a.out = y;
    return hip_status(moe::launch_w4_matvec(a, static_cast<hipStream_t>(stream)));
}

int moe_norm_in(const moe_norm* d, const void* x, const void* weight, const void* bias, void* y, void* stream)
{
    int rc = check_norm(d);
    if (rc) return rc;
    if (d->kind == MOE_NORM_NONE) return MOE_ERR_INVALID_ARG;
    if (d->T == 0) return MOE_OK;
    const size_t eb = type_bytes(d->dtype);
    if ((rc = check_norm_params(*d, false, weight, bias, nullptr, nullptr)) || (rc = need(x, eb)) || (rc = need(y, eb)))
        return rc;
    moe::NormArgs a = norm_args(*d, false);
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.out = y;
    return hip_status(moe::launch_norm_in(a, static_cast<hipStream_t>(stream)));
}

int moe_norm_out(const moe_norm* d, const void* f, const void* residual, const void* weight, const void* bias,
                 const void* gate, const uint64_t* rng, void* out, void* stream)
{
    int rc = check_norm(d);
    if (rc) return rc;
    if (d->T == 0) return MOE_OK;
    const size_t eb = type_bytes(d->dtype);
    if ((rc = check_norm_params(*d, true, weight, bias, gate, rng)) || (rc = need(f, eb)) || (rc = maybe(residual, eb)) ||
        (rc = need(out, eb)))
        return rc;
    moe::NormArgs a = norm_args(*d, true);
    a.x = f;
    a.res = residual;
    a.weight = weight;
    a.bias = bias;
    a.gate = gate;
    a.rng = rng;
    a.out = out;
    return hip_status(moe::launch_norm_out(a, static_cast<hipStream_t>(stream)));
}

int moe_norm_workspace_size(const moe_norm* d, size_t* bytes)
{
    int rc = check_norm(d);
    if (rc) return rc;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = norm_ws_bytes(*d);
    return MOE_OK;
}

int moe_norm_in_backward(const moe_norm* d, const void* x, const void* weight, const void* dy, const void* dres,
                         void* dx, float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_norm(d);
    if (rc) return rc;
    if (d->kind == MOE_NORM_NONE) return MOE_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if ((rc = maybe(dweight, 4)) || (rc = maybe(dbias, 4))) return rc;
    if (d->T == 0) {
        if ((rc = hip_status(moe::launch_zero16(dweight, 2ll * d->H, s)))) return rc;
        return hip_status(moe::launch_zero16(dbias, 2ll * d->H, s));
    }
    const size_t eb = type_bytes(d->dtype);
    if ((rc = check_norm_params(*d, false, weight, nullptr, nullptr, nullptr)) || (rc = need(x, eb)) ||
        (rc = need(dy, eb)) || (rc = maybe(dres, eb)) || (rc = need(dx, eb)) ||
        (rc = check_norm_ws(*d, workspace, workspace_bytes)))
        return rc;
    moe::NormArgs a = norm_args(*d, false);
    a.x = x;
    a.weight = weight;
    a.dout = dy;
    a.res = dres;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.part = static_cast<float*>(workspace);
    return hip_status(moe::launch_norm_in_backward(a, s));
}

int moe_norm_out_backward(const moe_norm* d, const void* f, const void* weight, const void* bias, const void* gate,
                          const uint64_t* rng, const void* dout, void* df, float* dweight, float* dbias, void* dgate,
                          void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_norm(d);
    if (rc) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (d->kind == MOE_NORM_NONE && (dweight || dbias)) return MOE_ERR_INVALID_ARG;
    if (d->gate == MOE_GATE_NONE && dgate) return MOE_ERR_INVALID_ARG;
    const size_t eb = type_bytes(d->dtype);
    if ((rc = maybe(dweight, 4)) || (rc = maybe(dbias, 4)) || (rc = maybe(dgate, d->gate == MOE_GATE_FULL ? eb : 4)))
        return rc;
    if (d->T == 0) {
        if ((rc = hip_status(moe::launch_zero16(dweight, 2ll * d->H, s)))) return rc;
        if ((rc = hip_status(moe::launch_zero16(dbias, 2ll * d->H, s)))) return rc;
        return d->gate == MOE_GATE_CHANNEL ? hip_status(moe::launch_zero16(dgate, 2ll * d->H, s)) : MOE_OK;
    }
    if ((rc = check_norm_params(*d, true, weight, bias, gate, rng)) || (rc = need(f, eb)) || (rc = need(dout, eb)) ||
        (rc = need(df, eb)) || (rc = check_norm_ws(*d, workspace, workspace_bytes)))
        return rc;
    moe::NormArgs a = norm_args(*d, true);
    a.x = f;
    a.weight = weight;
    a.bias = bias;
    a.gate = gate;
    a.rng = rng;
    a.dout = dout;
    a.dx = df;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dgate = dgate;
    a.part = static_cast<float*>(workspace);
    return hip_status(moe::launch_norm_out_backward(a, s));
}

}  // extern "C"
