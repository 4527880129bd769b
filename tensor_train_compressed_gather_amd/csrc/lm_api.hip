// lm_api.hip -- host side of the operators around the table (lookup, norm,
// blocknorm, ffn, xent, adamw, clip): argument checks before anything is enqueued, then the
// stream-ordered launches.  Nothing here allocates device memory, and no exception
// leaves.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>

#include "lm.h"

using namespace ttemb;

namespace {

bool bad_dtype(int32_t d) { return d != TT_EMB_DTYPE_FLOAT && d != TT_EMB_DTYPE_BFLOAT && d != TT_EMB_DTYPE_HALF; }
size_t dtype_size(int32_t d) { return d == TT_EMB_DTYPE_FLOAT ? 4 : 2; }
// Elements must lie at multiples of their size.
bool off_grid(const void *p, int32_t d) { return (reinterpret_cast<uintptr_t>(p) & (dtype_size(d) - 1)) != 0; }
bool bad_matrix(const void *p, int64_t ld, int64_t rows, int64_t cols, int32_t d)
{
    if (rows == 0) return false;
    return !p || off_grid(p, d) || ld < cols;
}
int check_ws(const void *ws, size_t have, size_t need)
{
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || have < need) return TT_EMB_ERR_WORKSPACE;
    return TT_EMB_OK;
}
int hip_status(hipError_t e) { return e == hipSuccess ? TT_EMB_OK : TT_EMB_ERR_HIP; }

constexpr int64_t kMaxRows = 0x7ffffffe;
constexpr int64_t kMaxLookupCols = 65536, kMaxNormCols = 16384, kMaxXentCols = 16384;
constexpr int64_t kMaxXentTiles = (int64_t)1 << 23;
constexpr int64_t kMaxFfnCols = 65536, kMaxFfnTiles = (int64_t)1 << 23;
constexpr int64_t kMaxClipValues = (int64_t)1 << 42;

int check_lookup(int64_t n, int64_t V, int64_t D, int32_t dtype)
{
    if (n < 0 || V <= 0 || D <= 0 || bad_dtype(dtype)) return TT_EMB_ERR_ARG;
    if (n > kMaxRows || V > kMaxRows || D > kMaxLookupCols) return TT_EMB_ERR_UNSUPPORTED;
    return TT_EMB_OK;
}

int check_norm(int64_t n, int64_t D, int32_t dtype, int32_t param_dtype)
{
    if (n < 0 || D <= 0 || bad_dtype(dtype)) return TT_EMB_ERR_ARG;
    if (param_dtype != TT_EMB_DTYPE_FLOAT && param_dtype != dtype) return TT_EMB_ERR_ARG;
    if (n > kMaxRows || D > kMaxNormCols) return TT_EMB_ERR_UNSUPPORTED;
    return TT_EMB_OK;
}

int check_xent(int64_t n, int64_t V, int64_t D, int32_t dtype)
{
    if (n < 0 || V <= 0 || D <= 0 || bad_dtype(dtype)) return TT_EMB_ERR_ARG;
    if (dtype == TT_EMB_DTYPE_HALF) return TT_EMB_ERR_UNSUPPORTED;
    if (n > kMaxRows || V > kMaxRows || D > kMaxXentCols) return TT_EMB_ERR_UNSUPPORTED;
    // tiles of the logits: the blocks of one launch stay below 2^24
    if (((n + 127) / 128) * ((V + 127) / 128) > kMaxXentTiles) return TT_EMB_ERR_UNSUPPORTED;
    return TT_EMB_OK;
}

int check_block(int64_t n, int64_t D, int32_t dtype, int32_t residual_dtype, int32_t param_dtype, int32_t kind)
{
    const int rc = check_norm(n, D, dtype, param_dtype);
    if (rc) return rc;
    if (residual_dtype != TT_EMB_DTYPE_FLOAT && residual_dtype != dtype) return TT_EMB_ERR_ARG;
    if ((kind & ~(TT_EMB_BLOCK_RMS | TT_EMB_BLOCK_POST | TT_EMB_BLOCK_GATE_ROWS)) != 0) return TT_EMB_ERR_ARG;
    return TT_EMB_OK;
}

// What both directions read, and its checks.
int block_args(BlockNormArgs &a, const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t n,
               int64_t D, int32_t dtype, int32_t residual_dtype, const void *gate, int64_t ld_gate,
               const void *post_gamma, const void *post_beta, const void *gamma, const void *beta,
               int32_t param_dtype, int32_t kind, float residual_scale, float block_scale)
{
    const int rc = check_block(n, D, dtype, residual_dtype, param_dtype, kind);
    if (rc) return rc;
    if (bad_matrix(x, ld_x, n, D, dtype) || bad_matrix(residual, ld_residual, n, D, residual_dtype))
        return TT_EMB_ERR_ARG;
    for (const void *p : {post_gamma, post_beta, gamma, beta})
        if (off_grid(p, param_dtype)) return TT_EMB_ERR_ARG;
    if ((kind & TT_EMB_BLOCK_RMS) && (beta || post_beta)) return TT_EMB_ERR_ARG;
    if (!(kind & TT_EMB_BLOCK_POST) && (post_gamma || post_beta)) return TT_EMB_ERR_ARG;
    if (kind & TT_EMB_BLOCK_GATE_ROWS) {
        if (bad_matrix(gate, ld_gate, n, D, dtype)) return TT_EMB_ERR_ARG;
    } else if (off_grid(gate, param_dtype)) {
        return TT_EMB_ERR_ARG;
    }
    a.x = x;
    a.residual = residual;
    a.gate = gate;
    a.ld_x = ld_x;
    a.ld_r = ld_residual;
    a.ld_gate = ld_gate;
    a.n = n;
    a.D = D;
    a.gate_rows = (kind & TT_EMB_BLOCK_GATE_ROWS) != 0;
    a.layer = !(kind & TT_EMB_BLOCK_RMS);
    a.post = (kind & TT_EMB_BLOCK_POST) != 0;
    a.gamma = gamma;
    a.beta = beta;
    a.post_gamma = post_gamma;
    a.post_beta = post_beta;
    a.param_dtype = param_dtype;
    a.scale_residual = residual_scale;
    a.scale_block = block_scale;
    return TT_EMB_OK;
}

int check_ffn(int64_t n, int64_t D, int64_t F, int32_t dtype, int32_t act)
{
    if (n < 0 || D <= 0 || F <= 0 || bad_dtype(dtype)) return TT_EMB_ERR_ARG;
    if (act != TT_EMB_ACT_SILU && act != TT_EMB_ACT_GELU && act != TT_EMB_ACT_GELU_TANH) return TT_EMB_ERR_ARG;
    if (n > kMaxRows || D > kMaxFfnCols || F > kMaxFfnCols) return TT_EMB_ERR_UNSUPPORTED;
    // tiles of p: the blocks of one launch stay below 2^24
    const int64_t wide = 2 * F > D ? 2 * F : D;
    if (((n + 127) / 128) * ((wide + 127) / 128) > kMaxFfnTiles) return TT_EMB_ERR_UNSUPPORTED;
    return TT_EMB_OK;
}

int check_clip(int32_t count, const int64_t *numel)
{
    if (count < 0 || (count > 0 && !numel)) return TT_EMB_ERR_ARG;
    int64_t all = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (numel[k] < 0) return TT_EMB_ERR_ARG;
        // the chunks of a launch and the partial sums of all stay below 2^31
        all += numel[k] > kMaxClipValues ? kMaxClipValues + 1 : numel[k];
        if (all > kMaxClipValues) return TT_EMB_ERR_UNSUPPORTED;
    }
    return TT_EMB_OK;
}

size_t clip_workspace(int32_t count, const int64_t *numel)
{
    return TT_EMB_STATUS_BYTES + round256((size_t)plan_clip(count, numel).parts * sizeof(double));
}

// Whether two of the tensors share memory: each is scaled once.
int check_apart(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel)
{
    struct Range {
        uintptr_t begin, end;
    };
    Range *r = new (std::nothrow) Range[count];
    if (!r) return TT_EMB_ERR_NOMEM;
    int32_t n = 0;
    for (int32_t k = 0; k < count; ++k) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(grads[k]);
        if (numel[k]) r[n++] = {p, p + (uintptr_t)numel[k] * dtype_size(dtypes[k])};
    }
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.begin < b.begin; });
    bool apart = true;
    for (int32_t k = 1; k < n; ++k) apart = apart && r[k - 1].end <= r[k].begin;
    delete[] r;
    return apart ? TT_EMB_OK : TT_EMB_ERR_ARG;
}

int clip(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel, double max_norm, double eps,
         float *norm, float *factor, bool scale, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_clip(count, numel);
    if (rc) return rc;
    if (!(max_norm >= 0.0) || !(eps >= 0.0) || !std::isfinite(eps)) return TT_EMB_ERR_ARG;
    if (off_grid(norm, TT_EMB_DTYPE_FLOAT) || off_grid(factor, TT_EMB_DTYPE_FLOAT)) return TT_EMB_ERR_ARG;
    if (count > 0 && (!grads || !dtypes)) return TT_EMB_ERR_ARG;
    for (int32_t k = 0; k < count; ++k) {
        if (bad_dtype(dtypes[k])) return TT_EMB_ERR_ARG;
        if (numel[k] && (!grads[k] || off_grid(grads[k], dtypes[k]))) return TT_EMB_ERR_ARG;
    }
    if (scale && (rc = check_apart(count, grads, dtypes, numel))) return rc;
    if ((rc = check_ws(ws, ws_bytes, clip_workspace(count, numel)))) return rc;
    const ClipBound b{max_norm, eps, norm, factor};
    return hip_status(launch_clip(count, grads, dtypes, numel, b, scale, static_cast<char *>(ws),
                                  (hipStream_t)stream));
}

} // namespace

extern "C" {

int tt_emb_poll_status(void *ws, void *stream)
{
    if (!ws) return TT_EMB_ERR_ARG;
    hipStream_t s = (hipStream_t)stream;
    int32_t err = 0;
    if (hipMemcpyAsync(&err, ws, sizeof(err), hipMemcpyDeviceToHost, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return TT_EMB_ERR_HIP;
    if (!err) return TT_EMB_OK;
    const int32_t zero = 0;
    if (hipMemcpyAsync(ws, &zero, sizeof(zero), hipMemcpyHostToDevice, s) != hipSuccess ||
        hipStreamSynchronize(s) != hipSuccess)
        return TT_EMB_ERR_HIP;
    return (err & STB_INDEX) ? TT_EMB_ERR_INDEX : TT_EMB_OK;
}

int tt_emb_lookup_workspace_size(int64_t n, int64_t V, int64_t D, size_t *bytes)
{
    if (!bytes) return TT_EMB_ERR_ARG;
    const int rc = check_lookup(n, V, D, TT_EMB_DTYPE_FLOAT);
    if (rc) return rc;
    *bytes = lookup_workspace(n, V, D);
    return TT_EMB_OK;
}

int tt_emb_lookup_forward(const void *weight, int64_t ld_weight, const int64_t *tokens, int64_t n, int64_t V,
                          int64_t D, int32_t dtype, float scale, void *out, int64_t ld_out, void *ws,
                          size_t ws_bytes, void *stream)
{
    int rc = check_lookup(n, V, D, dtype);
    if (rc) return rc;
    if (bad_matrix(weight, ld_weight, V, D, dtype) || bad_matrix(out, ld_out, n, D, dtype) || (n > 0 && !tokens))
        return TT_EMB_ERR_ARG;
    if ((rc = check_ws(ws, ws_bytes, TT_EMB_STATUS_BYTES))) return rc;
    LookupArgs a{};
    a.src = weight;
    a.ld_src = ld_weight;
    a.tokens = tokens;
    a.n = n;
    a.V = V;
    a.D = D;
    a.scale = scale;
    a.dst = out;
    a.ld_dst = ld_out;
    a.ws = static_cast<char *>(ws);
    return hip_status(launch_lookup_forward(a, dtype, (hipStream_t)stream));
}

int tt_emb_lookup_backward(const void *grad_out, int64_t ld_grad, const int64_t *tokens, int64_t n, int64_t V,
                           int64_t D, int32_t dtype, float scale, int64_t padding_idx, int32_t accumulate,
                           void *grad_weight, int64_t ld_weight, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_lookup(n, V, D, dtype);
    if (rc) return rc;
    if (bad_matrix(grad_weight, ld_weight, V, D, dtype) || bad_matrix(grad_out, ld_grad, n, D, dtype) ||
        (n > 0 && !tokens))
        return TT_EMB_ERR_ARG;
    if ((rc = check_ws(ws, ws_bytes, lookup_workspace(n, V, D)))) return rc;
    LookupArgs a{};
    a.src = grad_out;
    a.ld_src = ld_grad;
    a.tokens = tokens;
    a.n = n;
    a.V = V;
    a.D = D;
    a.scale = scale;
    a.dst = grad_weight;
    a.ld_dst = ld_weight;
    a.pad = padding_idx < 0 ? -1 : padding_idx;
    a.accumulate = accumulate != 0;
    a.ws = static_cast<char *>(ws);
    return hip_status(launch_lookup_backward(a, dtype, (hipStream_t)stream));
}

int tt_emb_norm_workspace_size(int64_t n, int64_t D, size_t *bytes)
{
    if (!bytes) return TT_EMB_ERR_ARG;
    const int rc = check_norm(n, D, TT_EMB_DTYPE_FLOAT, TT_EMB_DTYPE_FLOAT);
    if (rc) return rc;
    *bytes = norm_workspace(n, D);
    return TT_EMB_OK;
}

int tt_emb_norm_forward(const void *x, int64_t ld_x, int64_t n, int64_t D, int32_t dtype, const void *gamma,
                        const void *beta, int32_t param_dtype, float eps, void *y, int64_t ld_y, float *mean,
                        float *rstd, void *stream)
{
    const int rc = check_norm(n, D, dtype, param_dtype);
    if (rc) return rc;
    if (bad_matrix(x, ld_x, n, D, dtype) || bad_matrix(y, ld_y, n, D, dtype) || !(eps >= 0.f)) return TT_EMB_ERR_ARG;
    if (off_grid(gamma, param_dtype) || off_grid(beta, param_dtype)) return TT_EMB_ERR_ARG;
    NormArgs a{};
    a.x = x;
    a.ld_x = ld_x;
    a.n = n;
    a.D = D;
    a.gamma = gamma;
    a.beta = beta;
    a.param_dtype = param_dtype;
    a.eps = eps;
    a.y = y;
    a.ld_y = ld_y;
    a.mean = mean;
    a.rstd = rstd;
    return hip_status(launch_norm_forward(a, dtype, (hipStream_t)stream));
}

int tt_emb_norm_backward(const void *grad_y, int64_t ld_grad, const void *x, int64_t ld_x, int64_t n, int64_t D,
                         int32_t dtype, const void *gamma, int32_t param_dtype, const float *mean,
                         const float *rstd, void *grad_x, int64_t ld_grad_x, void *dgamma, void *dbeta, void *ws,
                         size_t ws_bytes, void *stream)
{
    int rc = check_norm(n, D, dtype, param_dtype);
    if (rc) return rc;
    if (bad_matrix(grad_y, ld_grad, n, D, dtype) || bad_matrix(x, ld_x, n, D, dtype) ||
        bad_matrix(grad_x, ld_grad_x, n, D, dtype) || (n > 0 && (!mean || !rstd)))
        return TT_EMB_ERR_ARG;
    if (off_grid(gamma, param_dtype) || off_grid(dgamma, param_dtype) || off_grid(dbeta, param_dtype))
        return TT_EMB_ERR_ARG;
    if ((rc = check_ws(ws, ws_bytes, norm_workspace(n, D)))) return rc;
    NormArgs a{};
    a.x = x;
    a.dy = grad_y;
    a.ld_x = ld_x;
    a.ld_dy = ld_grad;
    a.n = n;
    a.D = D;
    a.gamma = gamma;
    a.param_dtype = param_dtype;
    a.y = grad_x;
    a.ld_y = ld_grad_x;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.ws = static_cast<char *>(ws);
    return hip_status(launch_norm_backward(a, dtype, (hipStream_t)stream));
}

int tt_emb_block_workspace_size(int64_t n, int64_t D, size_t *bytes)
{
    if (!bytes) return TT_EMB_ERR_ARG;
    const int rc = check_norm(n, D, TT_EMB_DTYPE_FLOAT, TT_EMB_DTYPE_FLOAT);
    if (rc) return rc;
    *bytes = block_workspace(n, D);
    return TT_EMB_OK;
}

int tt_emb_block_forward(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t n,
                         int64_t D, int32_t dtype, int32_t residual_dtype, const void *gate, int64_t ld_gate,
                         const void *post_gamma, const void *post_beta, const void *gamma, const void *beta,
                         int32_t param_dtype, int32_t kind, float eps, float residual_scale, float block_scale,
                         void *y, int64_t ld_y, void *h, int64_t ld_h, float *stats, void *stream)
{
    BlockNormArgs a{};
    const int rc = block_args(a, x, ld_x, residual, ld_residual, n, D, dtype, residual_dtype, gate, ld_gate, post_gamma,
                              post_beta, gamma, beta, param_dtype, kind, residual_scale, block_scale);
    if (rc) return rc;
    if (bad_matrix(y, ld_y, n, D, dtype) || bad_matrix(h, ld_h, n, D, residual_dtype) || !(eps >= 0.f) ||
        off_grid(stats, TT_EMB_DTYPE_FLOAT))
        return TT_EMB_ERR_ARG;
    a.eps = eps;
    a.y = y;
    a.ld_y = ld_y;
    a.h = h;
    a.ld_h = ld_h;
    a.stats = stats;
    return hip_status(launch_block_forward(a, dtype, residual_dtype, (hipStream_t)stream));
}

int tt_emb_block_backward(const void *grad_y, int64_t ld_grad_y, const void *grad_h, int64_t ld_grad_h, const void *x,
                          int64_t ld_x, const void *residual, int64_t ld_residual, int64_t n, int64_t D,
                          int32_t dtype, int32_t residual_dtype, const void *gate, int64_t ld_gate,
                          const void *post_gamma, const void *post_beta, const void *gamma, int32_t param_dtype,
                          int32_t kind, float residual_scale, float block_scale, const float *stats, void *grad_x,
                          int64_t ld_grad_x, void *grad_residual, int64_t ld_grad_residual, void *grad_gate,
                          int64_t ld_grad_gate, void *dpost_gamma, void *dpost_beta, void *dgamma, void *dbeta,
                          void *ws, size_t ws_bytes, void *stream)
{
    BlockNormArgs a{};
    int rc = block_args(a, x, ld_x, residual, ld_residual, n, D, dtype, residual_dtype, gate, ld_gate, post_gamma,
                        post_beta, gamma, nullptr, param_dtype, kind, residual_scale, block_scale);
    if (rc) return rc;
    if (bad_matrix(grad_y, ld_grad_y, n, D, dtype) || (grad_h && bad_matrix(grad_h, ld_grad_h, n, D, residual_dtype)) ||
        bad_matrix(grad_x, ld_grad_x, n, D, dtype) ||
        bad_matrix(grad_residual, ld_grad_residual, n, D, residual_dtype) ||
        (n > 0 && (!stats || off_grid(stats, TT_EMB_DTYPE_FLOAT))))
        return TT_EMB_ERR_ARG;
    if (a.gate_rows ? bad_matrix(grad_gate, ld_grad_gate, n, D, dtype) : off_grid(grad_gate, param_dtype))
        return TT_EMB_ERR_ARG;
    for (const void *p : {dpost_gamma, dpost_beta, dgamma, dbeta})
        if (off_grid(p, param_dtype)) return TT_EMB_ERR_ARG;
    if (!a.post && (dpost_gamma || dpost_beta)) return TT_EMB_ERR_ARG;
    if ((rc = check_ws(ws, ws_bytes, block_workspace(n, D)))) return rc;
    a.grad_y = grad_y;
    a.ld_gy = ld_grad_y;
    a.grad_h = grad_h;
    a.ld_gh = ld_grad_h;
    a.stats = const_cast<float *>(stats);
    a.grad_x = grad_x;
    a.ld_gx = ld_grad_x;
    a.grad_r = grad_residual;
    a.ld_gr = ld_grad_residual;
    a.grad_gate = a.gate_rows ? grad_gate : nullptr;
    a.ld_gg = ld_grad_gate;
    a.sums[0] = dgamma;
    a.sums[1] = dbeta;
    a.sums[2] = dpost_gamma;
    a.sums[3] = dpost_beta;
    a.sums[4] = a.gate_rows ? nullptr : grad_gate;
    a.ws = static_cast<char *>(ws);
    return hip_status(launch_block_backward(a, dtype, residual_dtype, (hipStream_t)stream));
}

int tt_emb_ffn_workspace_size(int64_t n, int64_t D, int64_t F, int32_t dtype, int32_t what, size_t *bytes)
{
    if (!bytes || (what & ~(TT_EMB_FFN_GRAD | TT_EMB_FFN_ALIGNED))) return TT_EMB_ERR_ARG;
    const int rc = check_ffn(n, D, F, dtype, TT_EMB_ACT_SILU);
    if (rc) return rc;
    *bytes = ffn_workspace(n, D, F, dtype, what);
    return TT_EMB_OK;
}

int tt_emb_ffn_forward(const void *x, int64_t ld_x, const void *w_in, int64_t ld_in, const void *w_out, int64_t ld_out,
                       int64_t n, int64_t D, int64_t F, int32_t dtype, int32_t activation, float *pre, int64_t ld_pre,
                       void *y, int64_t ld_y, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_ffn(n, D, F, dtype, activation);
    if (rc) return rc;
    if (bad_matrix(x, ld_x, n, D, dtype) || bad_matrix(w_in, ld_in, 2 * F, D, dtype) ||
        bad_matrix(w_out, ld_out, D, F, dtype) || bad_matrix(y, ld_y, n, D, dtype) ||
        (pre && bad_matrix(pre, ld_pre, n, 2 * F, TT_EMB_DTYPE_FLOAT)))
        return TT_EMB_ERR_ARG;
    FfnArgs a{};
    a.x = x;
    a.w_in = w_in;
    a.w_out = w_out;
    a.ld_x = ld_x;
    a.ld_in = ld_in;
    a.ld_out = ld_out;
    a.n = n;
    a.D = D;
    a.F = F;
    a.act = activation;
    a.pre = pre;
    a.ld_pre = ld_pre;
    a.y = y;
    a.ld_y = ld_y;
    a.ws = static_cast<char *>(ws);
    if ((rc = check_ws(ws, ws_bytes, ffn_needs(a, dtype, false)))) return rc;
    return hip_status(launch_ffn_forward(a, dtype, (hipStream_t)stream));
}

int tt_emb_ffn_backward(const void *grad_y, int64_t ld_grad_y, const void *x, int64_t ld_x, const float *pre,
                        int64_t ld_pre, const void *w_in, int64_t ld_in, const void *w_out, int64_t ld_out, int64_t n,
                        int64_t D, int64_t F, int32_t dtype, int32_t activation, void *grad_x, int64_t ld_grad_x,
                        void *grad_w_in, int64_t ld_grad_in, void *grad_w_out, int64_t ld_grad_out, void *ws,
                        size_t ws_bytes, void *stream)
{
    int rc = check_ffn(n, D, F, dtype, activation);
    if (rc) return rc;
    if (bad_matrix(grad_y, ld_grad_y, n, D, dtype) || bad_matrix(x, ld_x, n, D, dtype) ||
        bad_matrix(pre, ld_pre, n, 2 * F, TT_EMB_DTYPE_FLOAT) || bad_matrix(w_in, ld_in, 2 * F, D, dtype) ||
        bad_matrix(w_out, ld_out, D, F, dtype) || bad_matrix(grad_x, ld_grad_x, n, D, dtype) ||
        bad_matrix(grad_w_in, ld_grad_in, 2 * F, D, dtype) || bad_matrix(grad_w_out, ld_grad_out, D, F, dtype))
        return TT_EMB_ERR_ARG;
    FfnArgs a{};
    a.gy = grad_y;
    a.ld_gy = ld_grad_y;
    a.x = x;
    a.w_in = w_in;
    a.w_out = w_out;
    a.ld_x = ld_x;
    a.ld_in = ld_in;
    a.ld_out = ld_out;
    a.n = n;
    a.D = D;
    a.F = F;
    a.act = activation;
    a.pre = const_cast<float *>(pre);
    a.ld_pre = ld_pre;
    a.gx = grad_x;
    a.ld_gx = ld_grad_x;
    a.gw_in = grad_w_in;
    a.ld_gin = ld_grad_in;
    a.gw_out = grad_w_out;
    a.ld_gout = ld_grad_out;
    a.ws = static_cast<char *>(ws);
    if ((rc = check_ws(ws, ws_bytes, ffn_needs(a, dtype, true)))) return rc;
    return hip_status(launch_ffn_backward(a, dtype, (hipStream_t)stream));
}

int tt_emb_xent_workspace_size(int64_t n, int64_t V, int64_t D, int32_t dtype, int32_t what, size_t *bytes,
                               size_t *least)
{
    if ((!bytes && !least) || (what & ~(TT_EMB_XENT_GRAD | TT_EMB_XENT_ALIGNED))) return TT_EMB_ERR_ARG;
    const int rc = check_xent(n, V, D, dtype);
    if (rc) return rc;
    xent_workspace(n, V, D, dtype, what, bytes, least);
    return TT_EMB_OK;
}

int tt_emb_xent_parts(int64_t n, int64_t V, int64_t D, int32_t dtype, int32_t what, size_t ws_bytes,
                      tt_emb_xent_part *parts, int64_t cap, int64_t *count, int32_t *slots)
{
    const int rc = check_xent(n, V, D, dtype);
    if (rc) return rc;
    if (n == 0 || (what & ~TT_EMB_XENT_ALIGNED) != TT_EMB_XENT_GRAD || cap < 0 || (cap > 0 && !parts) || !count || !slots) return TT_EMB_ERR_ARG;
    size_t least = 0;
    xent_workspace(n, V, D, dtype, what, nullptr, &least);
    if (ws_bytes < least) return TT_EMB_ERR_WORKSPACE;
    *count = xent_parts(n, V, D, dtype, what, ws_bytes, parts, cap, slots);
    return TT_EMB_OK;
}

int tt_emb_xent_forward(const void *hidden, int64_t ld_hidden, const void *weight, int64_t ld_weight,
                        const int64_t *targets, int64_t n, int64_t V, int64_t D, int32_t dtype,
                        int64_t ignore_index, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream)
{
    int rc = check_xent(n, V, D, dtype);
    if (rc) return rc;
    if (bad_matrix(hidden, ld_hidden, n, D, dtype) || bad_matrix(weight, ld_weight, V, D, dtype) ||
        (n > 0 && (!targets || !loss || !lse)))
        return TT_EMB_ERR_ARG;
    XentArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.ld_h = ld_hidden;
    a.ld_w = ld_weight;
    a.targets = targets;
    a.n = n;
    a.V = V;
    a.D = D;
    a.ignore = ignore_index;
    a.loss = loss;
    a.lse = lse;
    a.ws = static_cast<char *>(ws);
    a.ws_bytes = ws_bytes;
    if ((rc = check_ws(ws, ws_bytes, xent_least(a, dtype, false)))) return rc;
    return hip_status(launch_xent_forward(a, dtype, (hipStream_t)stream));
}

int tt_emb_xent_loss_grad(const void *hidden, int64_t ld_hidden, const void *weight, int64_t ld_weight,
                          const int64_t *targets, const float *grad_loss, int64_t n, int64_t V, int64_t D,
                          int32_t dtype, int64_t ignore_index, float *loss, float *lse, void *grad_hidden,
                          int64_t ld_grad_hidden, void *grad_weight, int64_t ld_grad_weight, void *ws,
                          size_t ws_bytes, void *stream)
{
    int rc = check_xent(n, V, D, dtype);
    if (rc) return rc;
    if (bad_matrix(hidden, ld_hidden, n, D, dtype) || bad_matrix(weight, ld_weight, V, D, dtype) ||
        bad_matrix(grad_hidden, ld_grad_hidden, n, D, dtype) ||
        bad_matrix(grad_weight, ld_grad_weight, V, D, dtype) ||
        (n > 0 && (!targets || !loss || !lse || !grad_loss)))
        return TT_EMB_ERR_ARG;
    XentArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.ld_h = ld_hidden;
    a.ld_w = ld_weight;
    a.targets = targets;
    a.grad_loss = grad_loss;
    a.n = n;
    a.V = V;
    a.D = D;
    a.ignore = ignore_index;
    a.loss = loss;
    a.lse = lse;
    a.dh = grad_hidden;
    a.ld_dh = ld_grad_hidden;
    a.dw = grad_weight;
    a.ld_dw = ld_grad_weight;
    a.ws = static_cast<char *>(ws);
    a.ws_bytes = ws_bytes;
    if ((rc = check_ws(ws, ws_bytes, xent_least(a, dtype, true)))) return rc;
    return hip_status(launch_xent_loss_grad(a, dtype, (hipStream_t)stream));
}

int tt_emb_adamw_state_size(int32_t count, const int64_t *numel, int64_t *elements)
{
    if (count < 0 || (count > 0 && !numel) || !elements) return TT_EMB_ERR_ARG;
    int64_t blocks = 0;
    for (int32_t k = 0; k < count; ++k) {
        if (numel[k] < 0) return TT_EMB_ERR_ARG;
        // one launch has fewer than 2^31 blocks of 256 elements over all tensors
        if (numel[k] > ((int64_t)1 << 38)) return TT_EMB_ERR_UNSUPPORTED;
        blocks += (numel[k] + kAdamBlock - 1) / kAdamBlock;
        if (blocks > 0x7fffffff - kAdamBlock) return TT_EMB_ERR_UNSUPPORTED;
    }
    *elements = blocks * kAdamBlock;
    return TT_EMB_OK;
}

int tt_emb_adamw_update(int32_t count, float *const *params, const void *const *grads, int32_t grad_dtype,
                        void *const *copies, const int64_t *numel, void *exp_avg, void *exp_avg_sq,
                        float *exp_avg_scale, float *exp_avg_sq_scale, int32_t state_bits, double lr,
                        double beta1, double beta2, double eps, double weight_decay, int64_t step, uint64_t seed,
                        void *stream)
{
    return tt_emb_adamw_update_scaled(count, params, grads, grad_dtype, nullptr, copies, numel, exp_avg, exp_avg_sq,
                                      exp_avg_scale, exp_avg_sq_scale, state_bits, lr, beta1, beta2, eps,
                                      weight_decay, step, seed, stream);
}

int tt_emb_adamw_update_scaled(int32_t count, float *const *params, const void *const *grads, int32_t grad_dtype,
                               const float *grad_scale, void *const *copies, const int64_t *numel, void *exp_avg,
                               void *exp_avg_sq, float *exp_avg_scale, float *exp_avg_sq_scale, int32_t state_bits,
                               double lr, double beta1, double beta2, double eps, double weight_decay, int64_t step,
                               uint64_t seed, void *stream)
{
    int64_t elements = 0;
    const int rc = tt_emb_adamw_state_size(count, numel, &elements);
    if (rc) return rc;
    if (bad_dtype(grad_dtype) || (state_bits != 32 && state_bits != 8) || step < 1) return TT_EMB_ERR_ARG;
    if (!(lr >= 0.0) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !((float)eps >= FLT_MIN) ||
        !(weight_decay >= 0.0))
        return TT_EMB_ERR_ARG;
    if (off_grid(grad_scale, TT_EMB_DTYPE_FLOAT)) return TT_EMB_ERR_ARG;
    if (elements == 0) return TT_EMB_OK;
    if (!params || !grads) return TT_EMB_ERR_ARG;
    for (int32_t k = 0; k < count; ++k) {
        if (numel[k] == 0) continue;
        if (!params[k] || off_grid(params[k], TT_EMB_DTYPE_FLOAT) || !grads[k] || off_grid(grads[k], grad_dtype))
            return TT_EMB_ERR_ARG;
        if (copies && (!copies[k] || off_grid(copies[k], TT_EMB_DTYPE_BFLOAT))) return TT_EMB_ERR_ARG;
    }
    for (const void *p : {(const void *)exp_avg, (const void *)exp_avg_sq})
        if (!p || (reinterpret_cast<uintptr_t>(p) & 15u) != 0) return TT_EMB_ERR_ARG;
    if (state_bits == 8 && (!exp_avg_scale || !exp_avg_sq_scale || off_grid(exp_avg_scale, TT_EMB_DTYPE_FLOAT) ||
                            off_grid(exp_avg_sq_scale, TT_EMB_DTYPE_FLOAT)))
        return TT_EMB_ERR_ARG;
    AdamTable t{};
    t.key = (uint32_t)(seed * 0x9E3779B1u) ^ (uint32_t)((uint64_t)step * 0x85EBCA77u);
    // in 64 bits, rounded once: 1 - beta in 32 bits would be off by 1e-6 of itself
    t.beta1 = (float)beta1;
    t.one_minus_beta1 = (float)(1.0 - beta1);
    t.beta2 = (float)beta2;
    t.one_minus_beta2 = (float)(1.0 - beta2);
    t.decay = (float)(1.0 - lr * weight_decay);
    t.size = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
    t.root = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
    t.eps = (float)eps;
    t.m = exp_avg;
    t.v = exp_avg_sq;
    t.m_scale = exp_avg_scale;
    t.v_scale = exp_avg_sq_scale;
    t.g_scale = grad_scale;
    return hip_status(launch_adamw(t, count, params, grads, grad_dtype, copies, numel, state_bits,
                                   (hipStream_t)stream));
}

int tt_emb_clip_workspace_size(int32_t count, const int64_t *numel, size_t *bytes)
{
    if (!bytes) return TT_EMB_ERR_ARG;
    const int rc = check_clip(count, numel);
    if (rc) return rc;
    *bytes = clip_workspace(count, numel);
    return TT_EMB_OK;
}

int tt_emb_clip_norm(int32_t count, const void *const *grads, const int32_t *dtypes, const int64_t *numel,
                     double max_norm, double eps, float *norm, float *factor, void *ws, size_t ws_bytes, void *stream)
{
    return clip(count, const_cast<void *const *>(grads), dtypes, numel, max_norm, eps, norm, factor, false, ws,
                ws_bytes, stream);
}

int tt_emb_clip_scale(int32_t count, void *const *grads, const int32_t *dtypes, const int64_t *numel,
                      double max_norm, double eps, float *norm, float *factor, void *ws, size_t ws_bytes, void *stream)
{
    return clip(count, grads, dtypes, numel, max_norm, eps, norm, factor, true, ws, ws_bytes, stream);
}

} // extern "C"
