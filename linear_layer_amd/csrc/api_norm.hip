// The C ABI of the residual norms: argument checks, then the launches on the
// caller's stream. Nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include <math.h>

#include "linear_layer.h"
#include "host.hpp"
#include "lowp.hpp"

using namespace ll;
using namespace ll::host;

namespace {

// A matrix argument: null or M rows of N elements of `elem` bytes, ld apart.
struct Mat {
    const void *p;
    int ld, elem;
    Range range(int M, int N) const { return {p, p != nullptr ? span(M, N, ld, elem) : 0}; }
    bool ok(int M, int N) const
    {
        return p == nullptr || (aligned(p, elem) && range(M, N).bytes >= 0);
    }
    bool ld_ok(int N) const { return p == nullptr || ld >= (N > 1 ? N : 1); }
    bool same(const Mat &o) const { return p != nullptr && p == o.p && ld == o.ld; }
};

Range vec(const void *p, int N) { return {p, p != nullptr ? (int64_t)N * 4 : 0}; }

}  // namespace

extern "C" {

int rmsnorm_residual(int M, int N, int type, const float *Y, int ldy, const float *w_post, const float *gate,
                     float alpha, const void *X, int ldx, const float *w_pre, float eps, void *XO, int ldxo, void *H,
                     int ldh, void *stream)
{
    const int es = type_bytes(type);
    if (es == 0 || M < 0 || N < 0 || !(eps >= 0.0f) || isinf(eps))
        return LL_ERR_INVALID_VALUE;
    const Mat y{Y, ldy, 4}, x{X, ldx, es}, xo{XO, ldxo, es}, h{H, ldh, es};
    if (!y.ld_ok(N) || !x.ld_ok(N) || !xo.ld_ok(N) || !h.ld_ok(N))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || N == 0)
        return LL_OK;
    if (X == nullptr || (XO == nullptr && H == nullptr) || !y.ok(M, N) || !x.ok(M, N) || !xo.ok(M, N) || !h.ok(M, N) ||
        !aligned(w_post, 4) || !aligned(gate, 4) || !aligned(w_pre, 4))
        return LL_ERR_INVALID_VALUE;
    // x' may be written over x itself; nothing else may meet an output
    const Range out[2] = {xo.range(M, N), h.range(M, N)};
    const Range in[4] = {y.range(M, N), vec(w_post, N), vec(gate, N), vec(w_pre, N)};
    const Range xr = x.range(M, N);
    if (any_overlap(out, 2, in, 4) || overlap(out[1], xr) || (!xo.same(x) && overlap(out[0], xr)))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    const NormParams p{Y, w_post, gate, w_pre, X, XO, H, ldy, ldx, ldxo, ldh, M, N, alpha, eps};
    return status(launch_rmsnorm_residual(type, p, static_cast<hipStream_t>(stream)));
}

int64_t ll_rmsnorm_grad_workspace_size(int M, int N)
{
    return M < 0 || N < 0 ? -1 : rmsnorm_grad_workspace(M, N);
}

int rmsnorm_residual_grad(int M, int N, int type, const void *DXO, int lddxo, const void *DH, int lddh,
                          const float *Y, int ldy, const float *w_post, const float *gate, float alpha, const void *X,
                          int ldx, const float *w_pre, float eps, float *DY, int lddy, void *DX, int lddx,
                          float *dgate, float *dw_post, float *dw_pre, void *workspace, int64_t workspace_bytes,
                          void *stream)
{
    const int es = type_bytes(type);
    if (es == 0 || M < 0 || N < 0 || !(eps >= 0.0f) || isinf(eps) || workspace_bytes < 0)
        return LL_ERR_INVALID_VALUE;
    const Mat y{Y, ldy, 4}, x{X, ldx, es}, dxo{DXO, lddxo, es}, dh{DH, lddh, es}, dy{DY, lddy, 4}, dx{DX, lddx, es};
    if (!y.ld_ok(N) || !x.ld_ok(N) || !dxo.ld_ok(N) || !dh.ld_ok(N) || !dy.ld_ok(N) || !dx.ld_ok(N))
        return LL_ERR_INVALID_VALUE;
    if (N == 0)
        return LL_OK;
    if (!aligned(w_post, 4) || !aligned(gate, 4) || !aligned(w_pre, 4) || !aligned(dgate, 4) || !aligned(dw_post, 4) ||
        !aligned(dw_pre, 4))
        return LL_ERR_INVALID_VALUE;
    if (M > 0 && (X == nullptr || (DXO == nullptr && DH == nullptr) || (DY != nullptr && Y == nullptr) ||
                  (Y == nullptr && (dgate != nullptr || dw_post != nullptr)) || !y.ok(M, N) || !x.ok(M, N) ||
                  !dxo.ok(M, N) || !dh.ok(M, N) || !dy.ok(M, N) || !dx.ok(M, N)))
        return LL_ERR_INVALID_VALUE;
    const int64_t need = rmsnorm_grad_workspace(M, N);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
        return LL_ERR_INVALID_VALUE;
    // dx may be written over dx'; nothing else may meet an output
    const Range out[6] = {dy.range(M, N), vec(dgate, N), vec(dw_post, N), vec(dw_pre, N), {workspace, need},
                          dx.range(M, N)};
    const Range in[6] = {y.range(M, N), vec(w_post, N), vec(gate, N), vec(w_pre, N), x.range(M, N), dh.range(M, N)};
    const Range dxor = dxo.range(M, N);
    if (any_overlap(out, 6, in, 6) || any_overlap(out, 5, &dxor, 1) || (!dx.same(dxo) && overlap(out[5], dxor)))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    const NormGradParams p{Y,   w_post, gate, w_pre, X,     DXO,  DH,   DY,   DX, dgate, dw_post, dw_pre, nullptr,
                           ldy, ldx,    lddxo, lddh, lddy,  lddx, M,    N,    alpha, eps,  0.0f};
    return status(launch_rmsnorm_grad(type, p, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
