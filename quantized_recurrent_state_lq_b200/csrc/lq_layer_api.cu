// lq_layer_api.cu -- the C ABI of the recurrent layer's operators
// (include/lq_state.h): argument checks, then one launch call.  Everything is
// validated on the host first; nothing is launched on error.
#include <math.h>

#include "../../include/lq_state.h"
#include "lq_layer.h"

namespace {

using lq::Rows;

int rc_of(cudaError_t e) { return e == cudaSuccess ? LQ_OK : LQ_ERR_CUDA; }

bool is_dtype(int32_t t) { return t == LQ_F32 || t == LQ_BF16 || t == LQ_F16; }
int size_of(int32_t t) { return t == LQ_F32 ? 4 : 2; }

bool misaligned(const void *p, int a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Token rows as bytes: n rows of `width` bytes, `stride` bytes apart.
struct Span {
    uintptr_t p;
    int64_t n, width, stride;
};

Span rows_of(const void *p, int64_t n, int64_t width, int64_t ld, int size) {
    return {reinterpret_cast<uintptr_t>(p), n, width * size, ld * size};
}
Span offsets(const Rows &r) {
    return {reinterpret_cast<uintptr_t>(r.cu), 1, ((int64_t)r.B + 1) * 4, ((int64_t)r.B + 1) * 4};
}
Span flat(const void *p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), bytes > 0 ? 1 : 0, bytes, bytes}; }

// Whether two arrays may share bytes.  Apart in memory, or different columns of
// the same rows (equal strides, the columns disjoint): they do not.
bool overlap(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
    const uintptr_t ae = a.p + (uintptr_t)((a.n - 1) * a.stride + a.width);
    const uintptr_t be = b.p + (uintptr_t)((b.n - 1) * b.stride + b.width);
    if (ae <= b.p || be <= a.p) return false;
    if (a.stride != b.stride || a.stride <= 0) return true;
    const int64_t d = b.p >= a.p ? (int64_t)((b.p - a.p) % a.stride)
                                 : (a.stride - (int64_t)((a.p - b.p) % a.stride)) % a.stride;
    return d < a.width || d + b.width > a.stride;
}

bool same(const Span &a, const Span &b) { return a.p == b.p && a.stride == b.stride && a.width == b.width; }

// A row stride too small for its rows, or beyond any array (2^28 elements; the
// spans above then fit 64 bits).
bool bad_ld(int64_t ld, int64_t width) { return ld < width || ld > (1ll << 28); }

// The rows of a prompt batch.
int check_rows(int32_t B, int32_t rows, const int32_t *d_cu) {
    if (B < 1) return LQ_ERR_SHAPE;
    if (rows < 0 || rows > (1 << 30) || misaligned(d_cu, 4)) return LQ_ERR_INVALID_ARG;
    if (!d_cu && rows % B != 0) return LQ_ERR_SHAPE;
    return LQ_OK;
}

int check_conv(const lq_conv_config *c) {
    if (!c || !is_dtype(c->dtype)) return LQ_ERR_INVALID_ARG;
    if (c->act != LQ_ACT_NONE && c->act != LQ_ACT_SILU) return LQ_ERR_INVALID_ARG;
    if (c->B < 1 || c->B > (1 << 30) || c->C < 1) return LQ_ERR_SHAPE;   // (a sequence's number plus a batch's fits an int)
    if (c->K < 2 || c->K > LQ_CONV_MAX_TAPS || c->C > (1 << 22)) return LQ_ERR_UNSUPPORTED;
    return LQ_OK;
}

int check_ssm(const lq_ssm_config *c) {
    if (!c || !is_dtype(c->dtype) || (c->softplus != 0 && c->softplus != 1)) return LQ_ERR_INVALID_ARG;
    if (c->B < 1 || c->H < 1 || c->G < 1 || c->G > c->H || c->H % c->G != 0) return LQ_ERR_SHAPE;
    if ((int64_t)c->B * c->H > (1 << 27)) return LQ_ERR_SHAPE;
    if ((c->dk != 64 && c->dk != 128) || (c->dv != 64 && c->dv != 128)) return LQ_ERR_UNSUPPORTED;
    return LQ_OK;
}

lq::SsmArgs ssm_args(const lq_ssm_config *c, int32_t rows, const int32_t *d_cu) {
    lq::SsmArgs a{};
    a.r.cu = d_cu;
    a.r.B = c->B;
    a.r.rows = rows;
    a.H = c->H; a.G = c->G; a.dk = c->dk; a.dv = c->dv;
    a.softplus = c->softplus;
    a.fail_row = -1;
    return a;
}

// What the prompt and the single-token call check alike.
int check_ssm_arrays(const lq_ssm_config *c, const lq::SsmArgs &a) {
    const int64_t n = a.r.rows;
    if (!a.S_out || !a.A || (n > 0 && (!a.x || !a.dt || !a.Bm || !a.Cm || !a.y))) return LQ_ERR_INVALID_ARG;
    const int e = size_of(c->dtype);
    if (misaligned(a.x, e) || misaligned(a.dt, e) || misaligned(a.Bm, e) || misaligned(a.Cm, e) ||
        misaligned(a.y, e) || misaligned(a.A, 4) || misaligned(a.D, 4) || misaligned(a.dt_bias, 4) ||
        misaligned(a.S0, 16) || misaligned(a.S_out, 16))
        return LQ_ERR_INVALID_ARG;
    const int64_t wx = (int64_t)c->H * c->dv, wb = (int64_t)c->G * c->dk;
    if (n > 0 && (bad_ld(a.ldx, wx) || bad_ld(a.ldy, wx) || bad_ld(a.lddt, c->H) || bad_ld(a.ldb, wb) || bad_ld(a.ldc, wb)))
        return LQ_ERR_SHAPE;
    const int64_t sb = (int64_t)c->B * c->H * c->dk * c->dv * 4;
    const Span in[] = {rows_of(a.x, n, wx, a.ldx, e),   rows_of(a.dt, n, c->H, a.lddt, e),
                       rows_of(a.Bm, n, wb, a.ldb, e),  rows_of(a.Cm, n, wb, a.ldc, e),
                       flat(a.A, (int64_t)c->H * 4),    flat(a.D, (int64_t)c->H * 4),
                       flat(a.dt_bias, (int64_t)c->H * 4), offsets(a.r)};
    const Span y = rows_of(a.y, n, wx, a.ldy, e), S = flat(a.S_out, sb), S0 = flat(a.S0, sb);
    for (const Span &i : in)
        if (overlap(i, y) || overlap(i, S)) return LQ_ERR_INVALID_ARG;
    if (overlap(y, S) || overlap(y, S0) || (overlap(S, S0) && a.S0 != a.S_out)) return LQ_ERR_INVALID_ARG;
    return LQ_OK;
}

int check_norm(const lq_norm_config *c, bool in) {
    if (!c || !is_dtype(c->dtype)) return LQ_ERR_INVALID_ARG;
    if (c->x_dtype != c->dtype && (in || c->x_dtype != LQ_F32)) return LQ_ERR_INVALID_ARG;
    if (!(c->eps > 0.0f) || !isfinite(c->eps) || c->rows < 0) return LQ_ERR_INVALID_ARG;
    if ((c->w_groups != 0 && c->w_groups != 1) || (c->gate_first != 0 && c->gate_first != 1)) return LQ_ERR_INVALID_ARG;
    if (c->G < 1 || c->D < 1 || (in && c->G != 1)) return LQ_ERR_SHAPE;
    if (c->D > LQ_NORM_MAX_D || (int64_t)c->G * c->D > (1 << 28) || (int64_t)c->rows * c->G > (1ll << 31) - 1)
        return LQ_ERR_UNSUPPORTED;
    return LQ_OK;
}

// An output of a norm may be exactly one of its inputs, or apart from it.
bool clash(const Span &out, const Span &in, bool same_type) {
    return overlap(out, in) && !(same_type && same(out, in));
}

int check_norm_arrays(const lq_norm_config *c, const lq::NormArgs &a, bool in) {
    const int64_t n = c->rows, w = (int64_t)c->G * c->D;
    const int e = size_of(c->dtype), ex = size_of(c->x_dtype);
    if (!a.w || (n > 0 && (!a.x || !a.y))) return LQ_ERR_INVALID_ARG;
    if (misaligned(a.x, ex) || misaligned(a.z, e) || misaligned(a.res, e) || misaligned(a.h, e) ||
        misaligned(a.y, e) || misaligned(a.w, 4) || misaligned(a.dscale, 4))
        return LQ_ERR_INVALID_ARG;
    if (n > 0 && (bad_ld(a.ldx, w) || bad_ld(a.ldy, w) || (a.z && bad_ld(a.ldz, w)) || (a.res && bad_ld(a.ldres, w)) ||
                  (a.h && bad_ld(a.ldh, w))))
        return LQ_ERR_SHAPE;
    const Span x = rows_of(a.x, n, w, a.ldx, ex), z = rows_of(a.z, n, w, a.ldz, e),
               res = rows_of(a.res, n, w, a.ldres, e), h = rows_of(a.h, n, w, a.ldh, e),
               y = rows_of(a.y, n, w, a.ldy, e);
    const Span wt = flat(a.w, (a.w_groups ? w : c->D) * 4), sc = flat(a.dscale, w * 4);
    const bool xt = c->x_dtype == c->dtype;
    for (const Span &o : {h, y})
        if (clash(o, x, xt) || clash(o, z, true) || clash(o, res, true) || overlap(o, wt) || overlap(o, sc))
            return LQ_ERR_INVALID_ARG;
    if (in && overlap(h, y)) return LQ_ERR_INVALID_ARG;
    return LQ_OK;
}

lq::NormArgs norm_args(const lq_norm_config *c, const void *x, int64_t ldx, const float *w, const void *res,
                       int64_t ldres, const float *dscale, void *y, int64_t ldy) {
    lq::NormArgs a{};
    a.rows = c->rows;
    a.G = c->G; a.D = c->D;
    a.eps = c->eps;
    a.x = x; a.ldx = ldx;
    a.w = w; a.w_groups = c->w_groups;
    a.act = c->act == LQ_ACT_SIGMOID;
    a.gate_first = c->gate_first;
    a.res = res; a.ldres = res ? ldres : 0;
    a.scale = c->scale; a.dscale = dscale;
    a.y = y; a.ldy = ldy;
    return a;
}

int ssm_prefill(const lq_ssm_config *cfg, int32_t rows, const int32_t *d_cu, const void *d_x, int64_t ldx,
                const void *d_dt, int64_t lddt, const float *d_A, const void *d_Bm, int64_t ldb, const void *d_Cm,
                int64_t ldc, const float *d_D, const float *d_dt_bias, const float *d_S0, float *d_S_out, void *d_y,
                int64_t ldy, void *d_ws, size_t ws_bytes, int64_t fail_row, void *stream) {
    int rc = check_ssm(cfg);
    if (!rc) rc = check_rows(cfg->B, rows, d_cu);
    if (rc) return rc;
    lq::SsmArgs a = ssm_args(cfg, rows, d_cu);
    a.x = d_x; a.ldx = ldx; a.dt = d_dt; a.lddt = lddt;
    a.Bm = d_Bm; a.ldb = ldb; a.Cm = d_Cm; a.ldc = ldc;
    a.A = d_A; a.D = d_D; a.dt_bias = d_dt_bias;
    a.S0 = d_S0; a.S_out = d_S_out; a.y = d_y; a.ldy = ldy;
    a.fail_row = fail_row;
    rc = check_ssm_arrays(cfg, a);
    if (rc) return rc;
    const size_t need = lq_ssm_workspace_bytes(cfg, rows);
    if (need > 0) {
        if (!d_ws || misaligned(d_ws, 256) || ws_bytes < need) return LQ_ERR_WORKSPACE;
        const int e = size_of(cfg->dtype);
        const int64_t wx = (int64_t)cfg->H * cfg->dv, wb = (int64_t)cfg->G * cfg->dk;
        const int64_t sb = (int64_t)cfg->B * cfg->H * cfg->dk * cfg->dv * 4;
        const Span ws = flat(d_ws, (int64_t)need);
        const Span other[] = {rows_of(d_x, rows, wx, ldx, e),  rows_of(d_dt, rows, cfg->H, lddt, e),
                              rows_of(d_Bm, rows, wb, ldb, e), rows_of(d_Cm, rows, wb, ldc, e),
                              rows_of(d_y, rows, wx, ldy, e),  flat(d_S0, sb), flat(d_S_out, sb),
                              flat(d_A, (int64_t)cfg->H * 4),  flat(d_D, (int64_t)cfg->H * 4),
                              flat(d_dt_bias, (int64_t)cfg->H * 4), offsets(a.r)};
        for (const Span &o : other)
            if (overlap(ws, o)) return LQ_ERR_INVALID_ARG;
        a.ws = static_cast<float *>(d_ws);
    }
    return rc_of(lq::launch_ssm_prefill(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int lq_conv_prefill(const lq_conv_config *cfg, int32_t rows, const int32_t *d_cu, const void *d_x, int64_t ldx,
                    const float *d_w, const float *d_bias, const void *d_state0, void *d_state_out, void *d_y,
                    int64_t ldy, void *stream) {
    int rc = check_conv(cfg);
    if (!rc) rc = check_rows(cfg->B, rows, d_cu);
    if (rc) return rc;
    if (!d_w || (rows > 0 && (!d_x || !d_y))) return LQ_ERR_INVALID_ARG;
    const int e = size_of(cfg->dtype);
    if (misaligned(d_x, e) || misaligned(d_y, e) || misaligned(d_state0, e) || misaligned(d_state_out, e) ||
        misaligned(d_w, 4) || misaligned(d_bias, 4))
        return LQ_ERR_INVALID_ARG;
    if (rows > 0 && (bad_ld(ldx, cfg->C) || bad_ld(ldy, cfg->C))) return LQ_ERR_SHAPE;
    const int64_t sb = (int64_t)cfg->B * (cfg->K - 1) * cfg->C * e;
    const Span x = rows_of(d_x, rows, cfg->C, ldx, e), y = rows_of(d_y, rows, cfg->C, ldy, e);
    const Span s0 = flat(d_state0, sb), so = flat(d_state_out, sb);
    const Span w = flat(d_w, (int64_t)cfg->C * cfg->K * 4), bias = flat(d_bias, (int64_t)cfg->C * 4);
    lq::ConvArgs a{};
    a.r.cu = d_cu; a.r.B = cfg->B; a.r.rows = rows;
    for (const Span &o : {y, so})
        if (overlap(o, x) || overlap(o, w) || overlap(o, bias) || overlap(o, offsets(a.r))) return LQ_ERR_INVALID_ARG;
    if (overlap(y, s0) || overlap(y, so) || (overlap(s0, so) && d_state0 != d_state_out)) return LQ_ERR_INVALID_ARG;
    a.C = cfg->C; a.K = cfg->K; a.act = cfg->act;
    a.x = d_x; a.ldx = ldx; a.w = d_w; a.bias = d_bias;
    a.state0 = d_state0; a.state_out = d_state_out;
    a.y = d_y; a.ldy = ldy;
    return rc_of(lq::launch_conv_prefill(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
}

int lq_conv_step(const lq_conv_config *cfg, void *d_state, const void *d_x, int64_t ldx, const float *d_w,
                 const float *d_bias, void *d_y, int64_t ldy, void *stream) {
    const int rc = check_conv(cfg);
    if (rc) return rc;
    if (!d_state || !d_x || !d_w || !d_y) return LQ_ERR_INVALID_ARG;
    const int e = size_of(cfg->dtype);
    if (misaligned(d_x, e) || misaligned(d_y, e) || misaligned(d_state, e) || misaligned(d_w, 4) ||
        misaligned(d_bias, 4))
        return LQ_ERR_INVALID_ARG;
    if (bad_ld(ldx, cfg->C) || bad_ld(ldy, cfg->C)) return LQ_ERR_SHAPE;
    const Span x = rows_of(d_x, cfg->B, cfg->C, ldx, e), y = rows_of(d_y, cfg->B, cfg->C, ldy, e);
    const Span st = flat(d_state, (int64_t)cfg->B * (cfg->K - 1) * cfg->C * e);
    const Span w = flat(d_w, (int64_t)cfg->C * cfg->K * 4), bias = flat(d_bias, (int64_t)cfg->C * 4);
    for (const Span &o : {y, st})
        if (overlap(o, w) || overlap(o, bias)) return LQ_ERR_INVALID_ARG;
    if (overlap(st, x) || overlap(st, y) || (overlap(x, y) && !same(x, y))) return LQ_ERR_INVALID_ARG;
    lq::ConvArgs a{};
    a.r.B = cfg->B; a.r.rows = cfg->B;
    a.C = cfg->C; a.K = cfg->K; a.act = cfg->act;
    a.x = d_x; a.ldx = ldx; a.w = d_w; a.bias = d_bias;
    a.state_out = d_state;
    a.y = d_y; a.ldy = ldy;
    return rc_of(lq::launch_conv_step(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
}

size_t lq_ssm_workspace_bytes(const lq_ssm_config *cfg, int32_t rows) {
    if (check_ssm(cfg) != LQ_OK || rows < 0) return 0;
    return lq::ssm_ws_bytes(cfg->dtype, cfg->B, rows, cfg->H, cfg->G, cfg->dk, cfg->dv);
}

int lq_ssm_prefill(const lq_ssm_config *cfg, int32_t rows, const int32_t *d_cu, const void *d_x, int64_t ldx,
                   const void *d_dt, int64_t lddt, const float *d_A, const void *d_Bm, int64_t ldb, const void *d_Cm,
                   int64_t ldc, const float *d_D, const float *d_dt_bias, const float *d_S0, float *d_S_out, void *d_y,
                   int64_t ldy, void *d_ws, size_t ws_bytes, void *stream) {
    return ssm_prefill(cfg, rows, d_cu, d_x, ldx, d_dt, lddt, d_A, d_Bm, ldb, d_Cm, ldc, d_D, d_dt_bias, d_S0, d_S_out,
                       d_y, ldy, d_ws, ws_bytes, -1, stream);
}

int lq_selftest_ssm_wait(const lq_ssm_config *cfg, int32_t rows, const int32_t *d_cu, const void *d_x, int64_t ldx,
                         const void *d_dt, int64_t lddt, const float *d_A, const void *d_Bm, int64_t ldb,
                         const void *d_Cm, int64_t ldc, const float *d_D, const float *d_dt_bias, const float *d_S0,
                         float *d_S_out, void *d_y, int64_t ldy, void *d_ws, size_t ws_bytes, int32_t row,
                         void *stream) {
    if (row < 0 || row >= rows) return LQ_ERR_INVALID_ARG;
    if (cfg && cfg->dtype != LQ_BF16) return LQ_ERR_UNSUPPORTED;
    return ssm_prefill(cfg, rows, d_cu, d_x, ldx, d_dt, lddt, d_A, d_Bm, ldb, d_Cm, ldc, d_D, d_dt_bias, d_S0, d_S_out,
                       d_y, ldy, d_ws, ws_bytes, row, stream);
}

int lq_ssm_step(const lq_ssm_config *cfg, float *d_S, const void *d_x, int64_t ldx, const void *d_dt, int64_t lddt,
                const float *d_A, const void *d_Bm, int64_t ldb, const void *d_Cm, int64_t ldc, const float *d_D,
                const float *d_dt_bias, void *d_y, int64_t ldy, void *stream) {
    int rc = check_ssm(cfg);
    if (rc) return rc;
    lq::SsmArgs a = ssm_args(cfg, cfg->B, nullptr);
    a.x = d_x; a.ldx = ldx; a.dt = d_dt; a.lddt = lddt;
    a.Bm = d_Bm; a.ldb = ldb; a.Cm = d_Cm; a.ldc = ldc;
    a.A = d_A; a.D = d_D; a.dt_bias = d_dt_bias;
    a.S0 = d_S; a.S_out = d_S; a.y = d_y; a.ldy = ldy;
    rc = check_ssm_arrays(cfg, a);
    if (rc) return rc;
    return rc_of(lq::launch_ssm_step(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
}

int lq_norm_in(const lq_norm_config *cfg, const void *d_x, int64_t ldx, const float *d_w, const void *d_res,
               int64_t ldres, const float *d_scale, void *d_h, int64_t ldh, void *d_y, int64_t ldy, void *stream) {
    int rc = check_norm(cfg, true);
    if (rc) return rc;
    lq::NormArgs a = norm_args(cfg, d_x, ldx, d_w, d_res, ldres, d_scale, d_y, ldy);
    a.h = d_h; a.ldh = d_h ? ldh : 0;
    rc = check_norm_arrays(cfg, a, true);
    if (rc || cfg->rows == 0) return rc;
    return rc_of(lq::launch_norm_in(a, cfg->dtype, static_cast<cudaStream_t>(stream)));
}

int lq_norm_out(const lq_norm_config *cfg, const void *d_x, int64_t ldx, const float *d_w, const void *d_z, int64_t ldz,
                const void *d_res, int64_t ldres, const float *d_scale, void *d_y, int64_t ldy, void *stream) {
    int rc = check_norm(cfg, false);
    if (rc) return rc;
    if (d_z && cfg->act != LQ_ACT_SILU && cfg->act != LQ_ACT_SIGMOID) return LQ_ERR_INVALID_ARG;
    lq::NormArgs a = norm_args(cfg, d_x, ldx, d_w, d_res, ldres, d_scale, d_y, ldy);
    a.z = d_z; a.ldz = d_z ? ldz : 0;
    rc = check_norm_arrays(cfg, a, false);
    if (rc || cfg->rows == 0) return rc;
    return rc_of(lq::launch_norm_out(a, cfg->dtype, cfg->x_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
