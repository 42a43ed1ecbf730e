// gdn_layer_api.cu -- the C ABI of the layer operators (include/gdn.h): argument checks, all on the
// host before anything is enqueued, workspace layout, and dispatch to the kernels.
#include "gdn.h"
#include "gdn_layer.cuh"

#include <math.h>
#include <stdint.h>

namespace {

constexpr double kMaxElements = 1099511627776.0;   // 2^40
constexpr long long kMaxLd = 1LL << 40;
// Row and step counters are 32-bit ints that run past the last row by up to one round of a kernel (the
// norm's 608 x 8 warps, the convolution's 8 x 256 steps and the steps that it loads ahead).
constexpr double kMaxRows = 2147483648.0 - 65536.0;

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
size_t elem(int dtype) { return dtype == GDN_F32 ? 4 : 2; }
bool dtype_ok(int d) { return d == GDN_F32 || d == GDN_BF16; }
bool act_ok(int a) { return a == GDN_ACT_NONE || a == GDN_ACT_SILU || a == GDN_ACT_GELU; }

// A row stride: 0 selects the packed width; else at least the width.
int row_stride(long long ld, long long width, long long *out) {
    if (ld != 0 && ld < width) return GDN_ERR_INVALID_ARG;
    if (ld > kMaxLd) return GDN_ERR_UNSUPPORTED_SHAPE;
    *out = ld == 0 ? width : ld;
    return GDN_OK;
}

template <size_t N>
int packed_ok(const void *const (&ptrs)[N]) {
    for (const void *p : ptrs)
        if (p != nullptr && !aligned16(p)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}
template <size_t N>
int strided_ok(const void *const (&ptrs)[N], size_t e) {
    for (const void *p : ptrs)
        if (((uintptr_t)p & (e - 1)) != 0) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

int conv_plan(const gdn_conv_shape *s, gdn::ConvParams *p) {
    if (s == nullptr || s->B <= 0 || s->T <= 0 || s->C <= 0 || s->W <= 0 || s->ldx < 0) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || (s->act != GDN_ACT_NONE && s->act != GDN_ACT_SILU)) return GDN_ERR_INVALID_ARG;
    if (s->W > 4 || s->B > 65535 || s->C > (1 << 22)) return GDN_ERR_UNSUPPORTED_SHAPE;
    *p = {};
    const int rc = row_stride(s->ldx, s->C, &p->ldx);
    if (rc != GDN_OK) return rc;
    if ((double)s->B * s->T >= kMaxRows || (double)s->B * s->T * (double)p->ldx >= kMaxElements)
        return GDN_ERR_UNSUPPORTED_SHAPE;
    p->B = s->B; p->T = s->T; p->C = s->C; p->W = s->W; p->act = s->act;
    return GDN_OK;
}

size_t conv_ws(const gdn::ConvParams &p) { return up256((size_t)gdn::conv_bwd_slices(p) * (p.W + 1) * p.C * 4); }

int scan_plan(const gdn_scan_shape *s, gdn::ScanParams *p, bool bwd) {
    if (s == nullptr || s->B <= 0 || s->T <= 0 || s->C <= 0 || s->N <= 0 || s->G <= 0) return GDN_ERR_INVALID_ARG;
    if (s->ldu < 0 || s->lddt < 0 || s->ldz < 0 || s->ldB < 0 || s->ldC < 0 || !dtype_ok(s->dtype)) return GDN_ERR_INVALID_ARG;
    if (s->N > 64 || s->C % s->G != 0 || s->B > 65535 || s->G > 65535 || s->C > (1 << 22)) return GDN_ERR_UNSUPPORTED_SHAPE;
    *p = {};
    const long long gn = (long long)s->G * s->N;
    int rc;
    if ((rc = row_stride(s->ldu, s->C, &p->ldu)) != GDN_OK || (rc = row_stride(s->lddt, s->C, &p->lddt)) != GDN_OK ||
        (rc = row_stride(s->ldz, s->C, &p->ldz)) != GDN_OK || (rc = row_stride(s->ldB, gn, &p->ldB)) != GDN_OK ||
        (rc = row_stride(s->ldC, gn, &p->ldC)) != GDN_OK)
        return rc;
    const double rows = (double)s->B * s->T;
    long long widest = p->ldu;
    for (long long ld : {p->lddt, p->ldz, p->ldB, p->ldC}) widest = ld > widest ? ld : widest;
    // the largest tensors: the strided inputs, the checkpoints, the backward's partial sums
    if (rows >= kMaxRows || rows * (double)widest >= kMaxElements || rows * s->C * s->N / 8.0 >= kMaxElements ||
        (double)s->B * s->C * 16 >= kMaxElements)
        return GDN_ERR_UNSUPPORTED_SHAPE;
    if ((double)s->B * s->G * gdn::scan_blocks(s->C, s->G, s->N) >= 2147483648.0 ||
        (double)s->B * s->C * s->N >= 2147483648.0 * 32.0 || rows * s->G * 2 * s->N + (double)s->C * (s->N + 2) >= 2147483647.0 * 32.0)
        return GDN_ERR_UNSUPPORTED_SHAPE;
    p->Bn = s->B; p->T = s->T; p->Cn = s->C; p->N = s->N; p->G = s->G;
    gdn::scan_split(p, bwd);
    return GDN_OK;
}

size_t scan_state_floats(const gdn::ScanParams &p) { return (size_t)p.Bn * p.Cn * p.N; }
size_t scan_seg_bytes(const gdn::ScanParams &p) {
    if (p.segs == 1) return 0;
    return up256(p.segs * scan_state_floats(p) * 4) + up256((size_t)p.segs * p.Bn * p.Cn * 4);
}
void scan_seg_place(gdn::ScanParams *p, char *ws) {
    p->seg_state = reinterpret_cast<float *>(ws);
    p->seg_sum = reinterpret_cast<float *>(ws + up256(p->segs * scan_state_floats(*p) * 4));
}
size_t scan_ckpt_total(const gdn::ScanParams &p) {
    return (size_t)((p.T + gdn::kScanTile - 1) / gdn::kScanTile) * scan_state_floats(p) * 4;
}
size_t scan_part_bc_bytes(const gdn::ScanParams &p) {
    return up256((size_t)gdn::scan_blocks(p.Cn, p.G, p.N) * p.Bn * p.T * p.G * 2 * p.N * 4);
}
size_t scan_part_c_bytes(const gdn::ScanParams &p) { return up256((size_t)p.segs * p.Bn * (p.N + 2) * p.Cn * 4); }
size_t scan_bwd_ws(const gdn::ScanParams &p) { return scan_seg_bytes(p) + scan_part_bc_bytes(p) + scan_part_c_bytes(p); }

int norm_plan(const gdn_norm_shape *s, gdn::NormParams *p) {
    if (s == nullptr || s->M <= 0 || s->G <= 0 || s->D <= 0 || s->ldx < 0 || s->ldz < 0) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || !act_ok(s->act) || !(s->eps > 0.f) || !isfinite(s->eps)) return GDN_ERR_INVALID_ARG;
    if (s->M >= kMaxRows || s->G > 65535 || s->D > 65536) return GDN_ERR_UNSUPPORTED_SHAPE;
    *p = {};
    const long long C = (long long)s->G * s->D;
    int rc;
    if ((rc = row_stride(s->ldx, C, &p->ldx)) != GDN_OK || (rc = row_stride(s->ldz, C, &p->ldz)) != GDN_OK) return rc;
    if ((double)s->M * (double)(p->ldx > p->ldz ? p->ldx : p->ldz) >= kMaxElements) return GDN_ERR_UNSUPPORTED_SHAPE;
    p->M = s->M; p->G = s->G; p->D = s->D; p->act = s->act; p->center = s->center != 0; p->eps = s->eps;
    p->slices = gdn::norm_bwd_slices(s->M, s->G, s->D, s->dtype);
    return GDN_OK;
}

size_t norm_ws(const gdn::NormParams &p) { return up256((size_t)p.slices * 2 * p.G * p.D * 4); }

int linear_plan(const gdn_linear_shape *s, gdn::LinearParams *p) {
    if (s == nullptr || s->M <= 0 || s->N <= 0 || s->K <= 0 || s->ldx < 0 || s->ldw < 0 || s->ldres < 0) return GDN_ERR_INVALID_ARG;
    if (!dtype_ok(s->dtype) || !act_ok(s->act)) return GDN_ERR_INVALID_ARG;
    *p = {};
    int rc;
    if ((rc = row_stride(s->ldx, s->K, &p->ldx)) != GDN_OK || (rc = row_stride(s->ldw, s->K, &p->ldw)) != GDN_OK ||
        (rc = row_stride(s->ldres, s->N, &p->ldres)) != GDN_OK)
        return rc;
    if ((double)s->M * (double)p->ldx >= kMaxElements || (double)s->N * (double)p->ldw >= kMaxElements ||
        (double)s->M * (double)p->ldres >= kMaxElements)
        return GDN_ERR_UNSUPPORTED_SHAPE;
    // with room to spare for 32-bit counters of rows, of tiles and of K steps times products, and for the
    // decode form's grid (N / 128 on the y axis)
    if (s->M > 4000000 || s->N > 4000000 || s->K > 4000000) return GDN_ERR_UNSUPPORTED_SHAPE;
    p->M = s->M; p->N = s->N; p->K = s->K; p->act = s->act;
    return GDN_OK;
}

// bf16 x and W with packed rows are read in place by TMA, so they are 16-byte aligned like every packed
// tensor. A single row has room for a copy, and the forward of few rows reads any address.
int linear_operands_ok(const gdn::LinearParams &p, int dtype, const void *x, const void *W, bool bwd) {
    if (dtype == GDN_F32 || (!bwd && p.M <= gdn::kLinearFewRows)) return GDN_OK;
    if ((p.ldx == p.K && p.M > 1 && !aligned16(x)) || (p.ldw == p.K && p.N > 1 && !aligned16(W))) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}

}  // namespace

extern "C" {

int gdn_conv_fwd(const gdn_conv_shape *shape, const void *x, const float *w, const float *bias, const void *s0,
                 const int *lens, void *y, void *s_T, void *stream) {
    gdn::ConvParams p;
    int rc = conv_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    if (!x || !w || !y) return GDN_ERR_INVALID_ARG;
    if (s_T != nullptr && s_T == s0 && p.T != 1) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({w, bias, s0, lens, y, s_T})) != GDN_OK || (rc = strided_ok({x}, elem(shape->dtype))) != GDN_OK) return rc;
    gdn::api_clear_error();
    p.x = x; p.w = w; p.bias = bias; p.s0 = s0; p.lens = lens; p.y = y; p.s_T = s_T;
    return gdn::api_cuda_status(gdn::launch_conv_fwd(p, shape->dtype, (cudaStream_t)stream));
}

size_t gdn_conv_bwd_workspace_bytes(const gdn_conv_shape *shape) {
    gdn::ConvParams p;
    return conv_plan(shape, &p) == GDN_OK ? conv_ws(p) : 0;
}

int gdn_conv_bwd(const gdn_conv_shape *shape, const void *x, const float *w, const float *bias, const void *s0,
                 const int *lens, const void *dy, const void *ds_T, void *dx, float *dw, float *dbias, void *ds0,
                 void *workspace, size_t workspace_bytes, void *stream) {
    gdn::ConvParams p;
    int rc = conv_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    if (!x || !w || !dy || !dx || !dw || !workspace) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({w, bias, s0, lens, dy, ds_T, dx, dw, dbias, ds0, workspace})) != GDN_OK ||
        (rc = strided_ok({x}, elem(shape->dtype))) != GDN_OK)
        return rc;
    if (workspace_bytes < conv_ws(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.x = x; p.w = w; p.bias = bias; p.s0 = s0; p.lens = lens; p.dy = dy; p.ds_T = ds_T;
    p.dx = dx; p.dw = dw; p.dbias = dbias; p.ds0 = ds0; p.part = static_cast<float *>(workspace);
    return gdn::api_cuda_status(gdn::launch_conv_bwd(p, shape->dtype, (cudaStream_t)stream));
}

size_t gdn_scan_ckpt_bytes(const gdn_scan_shape *shape) {
    gdn::ScanParams p;
    return scan_plan(shape, &p, false) == GDN_OK ? scan_ckpt_total(p) : 0;
}

size_t gdn_scan_fwd_workspace_bytes(const gdn_scan_shape *shape) {
    gdn::ScanParams p;
    return scan_plan(shape, &p, false) == GDN_OK ? scan_seg_bytes(p) : 0;
}

size_t gdn_scan_bwd_workspace_bytes(const gdn_scan_shape *shape) {
    gdn::ScanParams p;
    return scan_plan(shape, &p, true) == GDN_OK ? scan_bwd_ws(p) : 0;
}

int gdn_scan_fwd(const gdn_scan_shape *shape, const void *u, const void *dt, const float *A_log, const void *B,
                 const void *C, const float *D, const float *dt_bias, const void *z, const float *h0, const int *lens,
                 void *y, float *h_T, float *ckpt, size_t ckpt_bytes, void *workspace, size_t workspace_bytes, void *stream) {
    gdn::ScanParams p;
    int rc = scan_plan(shape, &p, false);
    if (rc != GDN_OK) return rc;
    if (!u || !dt || !A_log || !B || !C || !y || (scan_seg_bytes(p) > 0 && !workspace)) return GDN_ERR_INVALID_ARG;
    if (h_T != nullptr && h_T == h0 && p.T != 1) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({A_log, D, dt_bias, h0, lens, y, h_T, ckpt, workspace})) != GDN_OK ||
        (rc = strided_ok({u, dt, B, C, z}, elem(shape->dtype))) != GDN_OK)
        return rc;
    if (ckpt != nullptr && ckpt_bytes < scan_ckpt_total(p)) return GDN_ERR_BUFFER_TOO_SMALL;
    if (workspace_bytes < scan_seg_bytes(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.u = u; p.dt = dt; p.A_log = A_log; p.B = B; p.C = C; p.D = D; p.dt_bias = dt_bias; p.z = z; p.h0 = h0;
    p.lens = lens; p.y = y; p.h_T = h_T; p.ckpt = ckpt;
    scan_seg_place(&p, static_cast<char *>(workspace));
    return gdn::api_cuda_status(gdn::launch_scan_fwd(p, shape->dtype, (cudaStream_t)stream));
}

int gdn_scan_bwd(const gdn_scan_shape *shape, const void *u, const void *dt, const float *A_log, const void *B,
                 const void *C, const float *D, const float *dt_bias, const void *z, const int *lens, const float *ckpt,
                 size_t ckpt_bytes, const void *dy, const float *dh_T, void *du, void *ddt, float *dA_log, void *dB, void *dC,
                 float *dD, float *ddt_bias, void *dz, float *dh0, void *workspace, size_t workspace_bytes, void *stream) {
    gdn::ScanParams p;
    int rc = scan_plan(shape, &p, true);
    if (rc != GDN_OK) return rc;
    if (!u || !dt || !A_log || !B || !C || !ckpt || !dy || !du || !ddt || !dA_log || !dB || !dC || !workspace)
        return GDN_ERR_INVALID_ARG;
    if (dz != nullptr && z == nullptr) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({A_log, D, dt_bias, lens, ckpt, dy, dh_T, du, ddt, dA_log, dB, dC, dD, ddt_bias, dz, dh0, workspace})) !=
            GDN_OK ||
        (rc = strided_ok({u, dt, B, C, z}, elem(shape->dtype))) != GDN_OK)
        return rc;
    if (ckpt_bytes < scan_ckpt_total(p)) return GDN_ERR_BUFFER_TOO_SMALL;
    if (workspace_bytes < scan_bwd_ws(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.u = u; p.dt = dt; p.A_log = A_log; p.B = B; p.C = C; p.D = D; p.dt_bias = dt_bias; p.z = z; p.lens = lens;
    p.ckpt = const_cast<float *>(ckpt); p.dy = dy; p.dh_T = dh_T;
    p.du = du; p.ddt = ddt; p.dA_log = dA_log; p.dB = dB; p.dC = dC; p.dD = dD; p.ddt_bias = ddt_bias; p.dz = dz; p.dh0 = dh0;
    char *ws = static_cast<char *>(workspace);
    scan_seg_place(&p, ws);
    p.part_bc = reinterpret_cast<float *>(ws + scan_seg_bytes(p));
    p.part_c = reinterpret_cast<float *>(ws + scan_seg_bytes(p) + scan_part_bc_bytes(p));
    return gdn::api_cuda_status(gdn::launch_scan_bwd(p, shape->dtype, (cudaStream_t)stream));
}

int gdn_norm_fwd(const gdn_norm_shape *shape, const void *x, const float *w, const float *b, const void *z, void *y,
                 float *stats, void *stream) {
    gdn::NormParams p;
    int rc = norm_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    if (!x || !y) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({w, b, y, stats})) != GDN_OK || (rc = strided_ok({x, z}, elem(shape->dtype))) != GDN_OK) return rc;
    gdn::api_clear_error();
    p.x = x; p.w = w; p.b = b; p.z = z; p.y = y; p.stats = stats;
    return gdn::api_cuda_status(gdn::launch_norm_fwd(p, shape->dtype, (cudaStream_t)stream));
}

size_t gdn_norm_bwd_workspace_bytes(const gdn_norm_shape *shape) {
    gdn::NormParams p;
    return norm_plan(shape, &p) == GDN_OK ? norm_ws(p) : 0;
}

int gdn_norm_bwd(const gdn_norm_shape *shape, const void *x, const float *w, const float *b, const void *z,
                 const float *stats, const void *dy, void *dx, float *dw, float *db, void *dz, void *workspace,
                 size_t workspace_bytes, void *stream) {
    gdn::NormParams p;
    int rc = norm_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    if (!x || !stats || !dy || !dx || !workspace || (dz != nullptr && z == nullptr)) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({w, b, stats, dy, dx, dw, db, dz, workspace})) != GDN_OK ||
        (rc = strided_ok({x, z}, elem(shape->dtype))) != GDN_OK)
        return rc;
    if (workspace_bytes < norm_ws(p)) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.x = x; p.w = w; p.b = b; p.z = z; p.stats_in = stats; p.dy = dy; p.dx = dx; p.dw = dw; p.db = db; p.dz = dz;
    p.part = static_cast<float *>(workspace);
    return gdn::api_cuda_status(gdn::launch_norm_bwd(p, shape->dtype, (cudaStream_t)stream));
}

size_t gdn_linear_fwd_workspace_bytes(const gdn_linear_shape *shape) {
    gdn::LinearParams p;
    return linear_plan(shape, &p) == GDN_OK ? gdn::linear_fwd_workspace(p, shape->dtype) : 0;
}

size_t gdn_linear_bwd_workspace_bytes(const gdn_linear_shape *shape) {
    gdn::LinearParams p;
    return linear_plan(shape, &p) == GDN_OK ? gdn::linear_bwd_workspace(p, shape->dtype) : 0;
}

int gdn_linear_fwd(const gdn_linear_shape *shape, const void *x, const void *W, const void *bias, const void *res, void *y,
                   void *pre, void *workspace, size_t workspace_bytes, void *stream) {
    gdn::LinearParams p;
    int rc = linear_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    const size_t need = gdn::linear_fwd_workspace(p, shape->dtype);
    if (!x || !W || !y || (need > 0 && !workspace)) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({bias, y, pre, workspace})) != GDN_OK || (rc = strided_ok({x, W, res}, elem(shape->dtype))) != GDN_OK ||
        (rc = linear_operands_ok(p, shape->dtype, x, W, false)) != GDN_OK)
        return rc;
    if (workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.x = x; p.W = W; p.bias = bias; p.res = res; p.y = y; p.pre = pre; p.ws = static_cast<char *>(workspace);
    if ((rc = gdn::api_device_status_address(&p.status)) != GDN_OK) return rc;
    return gdn::launch_linear_fwd(p, shape->dtype, (cudaStream_t)stream);
}

int gdn_linear_bwd(const gdn_linear_shape *shape, const void *x, const void *W, const void *pre, const void *dy, void *dx,
                   void *dW, void *dbias, void *workspace, size_t workspace_bytes, void *stream) {
    gdn::LinearParams p;
    int rc = linear_plan(shape, &p);
    if (rc != GDN_OK) return rc;
    const size_t need = gdn::linear_bwd_workspace(p, shape->dtype);
    if (!x || !W || !dy || (need > 0 && !workspace) || (shape->act != GDN_ACT_NONE && !pre)) return GDN_ERR_INVALID_ARG;
    if ((rc = packed_ok({pre, dy, dx, dW, dbias, workspace})) != GDN_OK || (rc = strided_ok({x, W}, elem(shape->dtype))) != GDN_OK ||
        (rc = linear_operands_ok(p, shape->dtype, x, W, true)) != GDN_OK)
        return rc;
    if (workspace_bytes < need) return GDN_ERR_WORKSPACE_TOO_SMALL;
    gdn::api_clear_error();
    p.x = x; p.W = W; p.pre_in = pre; p.dy = dy; p.dx = dx; p.dW = dW; p.dbias = dbias; p.ws = static_cast<char *>(workspace);
    if ((rc = gdn::api_device_status_address(&p.status)) != GDN_OK) return rc;
    return gdn::launch_linear_bwd(p, shape->dtype, (cudaStream_t)stream);
}

}  // extern "C"
