// The C ABI of the 16-bit layer, its gradients and the 8-bit format: argument checks, then
// the launches on the caller's stream. Nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include "host.hpp"
#include "linear16.hpp"
#include "linear_layer.h"

using namespace ll;
using namespace ll::host;

namespace {

// A matrix argument: null or rows of `elem`-byte elements, ld apart.
struct Mat {
    const void *p;
    int64_t ld;
    int elem;
    bool ld_ok(int64_t cols) const { return p == nullptr || ld >= (cols > 1 ? cols : 1); }
    Range range(int64_t rows, int64_t cols) const { return {p, p != nullptr ? span(rows, cols, ld, elem) : 0}; }
    bool ok(int64_t rows, int64_t cols) const { return p == nullptr || (aligned(p, elem) && range(rows, cols).bytes >= 0); }
    // every row in whole 16-byte pieces, on 16 bytes, and a tile of them in a buffer's 2 GiB
    bool vec(int64_t cols) const
    {
        return aligned(p, 16) && ld * elem % 16 == 0 && cols * elem % 16 == 0 && ld < (int64_t)1 << 21;
    }
    bool same(const Mat &o) const { return p != nullptr && p == o.p && ld == o.ld; }
};

// One matrix for each of n groups, `stride` elements apart: its range.
Range stack_range(const Mat &m, int64_t rows, int64_t cols, int64_t stride, int n)
{
    const Range one = m.range(rows, cols);
    int64_t more;
    if (m.p == nullptr || one.bytes <= 0 || n <= 1)
        return one;
    if (__builtin_mul_overflow((int64_t)(n - 1) * m.elem, stride, &more) || __builtin_add_overflow(one.bytes, more, &more))
        return {m.p, -1};
    return {m.p, more};
}

Range vec_range(const void *p, int64_t n) { return {p, p != nullptr ? n * 4 : 0}; }

bool type16(int type) { return type == LL_TYPE_F16 || type == LL_TYPE_BF16; }
// The type of an output beside 16-bit inputs of `type`.
bool out_type(int t, int type) { return t == type || t == LL_TYPE_F32; }

bool groups_ok(const int32_t *offsets, int groups)
{
    return offsets == nullptr ? groups == 1 : groups >= 0 && groups <= LL_MAX_GROUPS && aligned(offsets, 4);
}
Range groups_range(const int32_t *offsets, int groups) { return vec_range(offsets, (int64_t)groups + 1); }

// Of the sums of so many shares of an M x N result.
int64_t shares_bytes(int shares, int M, int N) { return shares > 1 ? (int64_t)shares * M * N * 4 : 0; }

int blocks_of(int cols) { return cols / 32 + (cols % 32 != 0); }

}  // namespace

extern "C" {

int mx8_quantize(int M, int K, int type, const void *X, int ldx, uint8_t *codes, int ldq, uint8_t *scales, int lds,
                 void *stream)
{
    const int es = type_bytes(type);
    const Mat x{X, ldx, es}, q{codes, ldq, 1}, sc{scales, lds, 1};
    if (es == 0 || M < 0 || K < 0 || !x.ld_ok(K) || !q.ld_ok(K) || !sc.ld_ok(blocks_of(K)))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || K == 0)
        return LL_OK;
    if (X == nullptr || codes == nullptr || scales == nullptr || !x.ok(M, K) || !q.ok(M, K) || !sc.ok(M, blocks_of(K)))
        return LL_ERR_INVALID_VALUE;
    const Range out[2] = {q.range(M, K), sc.range(M, blocks_of(K))}, in[1] = {x.range(M, K)};
    if (any_overlap(out, 2, in, 1))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    return status(launch_mx8_quantize(type, X, ldx, codes, ldq, scales, lds, M, K, static_cast<hipStream_t>(stream)));
}

int mx8_dequantize(int M, int K, const uint8_t *codes, int ldq, const uint8_t *scales, int lds, int type, void *Y, int ldy,
                   void *stream)
{
    const int es = type_bytes(type);
    const Mat y{Y, ldy, es}, q{codes, ldq, 1}, sc{scales, lds, 1};
    if (es == 0 || M < 0 || K < 0 || !y.ld_ok(K) || !q.ld_ok(K) || !sc.ld_ok(blocks_of(K)))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || K == 0)
        return LL_OK;
    if (Y == nullptr || codes == nullptr || scales == nullptr || !y.ok(M, K) || !q.ok(M, K) || !sc.ok(M, blocks_of(K)))
        return LL_ERR_INVALID_VALUE;
    const Range out[1] = {y.range(M, K)}, in[2] = {q.range(M, K), sc.range(M, blocks_of(K))};
    if (any_overlap(out, 1, in, 2))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    return status(launch_mx8_dequantize(type, codes, ldq, scales, lds, Y, ldy, M, K, static_cast<hipStream_t>(stream)));
}

const char *ll_linear16_chosen_kernel(int product, int M, int N, int K, int groups, int aligned, int num_cus)
{
    if (product < LL_L16_FORWARD || product > LL_L16_GRAD_WEIGHT || M <= 0 || N <= 0 || K <= 0 || groups <= 0 ||
        groups > LL_MAX_GROUPS || M > kL16Most || N > kL16Most || K > kL16Most)
        return "";
    return l16_kernel_name(product, M, N, K, groups, aligned != 0, num_cus > 0 ? num_cus : 256);
}

int64_t ll_linear16_workspace_size(int product, int M, int N, int K, int groups)
{
    if ((product != LL_L16_FORWARD && product != LL_L16_GRAD_INPUT) || M < 0 || N < 0 || K < 0 || groups < 0 ||
        groups > LL_MAX_GROUPS)
        return -1;
    if (M > kL16Most || N > kL16Most || K > kL16Most)   // (which no product takes)
        return 0;
    const Device dev = current_device();
    const int cus = dev.status == LL_OK ? dev.cus : 256;
    return shares_bytes(l16_shares(product, M, N, K, groups, cus), M, product == LL_L16_FORWARD ? N : K);
}

int linear16_nt(int M, int N, int K, int type, const uint16_t *X, int ldx, int groups, const int32_t *offsets,
                const uint16_t *W, int ldw, int64_t stride_w, const float *bias, int act, int ytype, const void *R, int ldr,
                void *Y, int ldy, uint16_t *Z, int ldz, uint8_t *ZQ, int ldzq, uint8_t *ZS, int ldzs, void *workspace,
                int64_t workspace_bytes, void *stream)
{
    if (!type16(type) || !out_type(ytype, type) || workspace_bytes < 0 || M < 0 || N < 0 || K < 0 || act < LL_ACT_NONE || act > LL_ACT_SILU ||
        !groups_ok(offsets, groups) || stride_w < 0 || (ZQ == nullptr) != (ZS == nullptr))
        return LL_ERR_INVALID_VALUE;
    const int es = type_bytes(ytype);
    const Mat x{X, ldx, 2}, w{W, ldw, 2}, r{R, ldr, es}, y{Y, ldy, es}, z{Z, ldz, 2}, zq{ZQ, ldzq, 1}, zs{ZS, ldzs, 1};
    const int nb = blocks_of(N);
    if (!x.ld_ok(K) || !w.ld_ok(K) || !r.ld_ok(N) || !y.ld_ok(N) || !z.ld_ok(N) || !zq.ld_ok(N) || !zs.ld_ok(nb))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || N == 0 || groups == 0)
        return LL_OK;
    const Range wr = stack_range(w, N, K, stride_w, groups);
    if (Y == nullptr || (K > 0 && (X == nullptr || W == nullptr)) || M > kL16Most || N > kL16Most || K > kL16Most ||
        !x.ok(M, K) || !w.ok(N, K) || wr.bytes < 0 || !r.ok(M, N) || !y.ok(M, N) || !z.ok(M, N) || !zq.ok(M, N) ||
        !zs.ok(M, nb) || !aligned(bias, 4))
        return LL_ERR_INVALID_VALUE;
    // y may be written over r itself; nothing else may meet an output
    const Range out[4] = {z.range(M, N), zq.range(M, N), zs.range(M, nb), y.range(M, N)};
    const Range in[4] = {x.range(M, K), wr, vec_range(bias, (int64_t)groups * N), groups_range(offsets, groups)};
    const Range rr = r.range(M, N);
    if (any_overlap(out, 4, in, 4) || any_overlap(out, 3, &rr, 1) || (!y.same(r) && overlap(out[3], rr)))
        return LL_ERR_INVALID_VALUE;
    if (workspace != nullptr && !aligned(workspace, 16))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    const int shares = workspace != nullptr ? l16_shares(L16_FWD, M, N, K, groups, dev.cus) : 1;
    const int64_t need = shares_bytes(shares, M, N);
    const Range ws = {workspace, need};
    if (need > 0 && (workspace_bytes < need || any_overlap(&ws, 1, in, 4) || any_overlap(&ws, 1, out, 4) || overlap(ws, rr)))
        return LL_ERR_INVALID_VALUE;
    L16Params p{};
    p.ws = static_cast<float *>(workspace);
    p.shares = shares;
    p.A = X;
    p.B = W;
    p.C = Y;
    p.bias = bias;
    p.R = R;
    p.Z = Z;
    p.ZQ = ZQ;
    p.ZS = ZS;
    p.lda = ldx, p.ldb = ldw, p.ldc = ldy, p.ldr = ldr, p.ldz = ldz, p.ldzq = ldzq, p.ldzs = ldzs;
    p.stride_b = stride_w;
    p.groups = Groups{offsets, groups};
    p.M = M, p.N = N, p.K = K;
    p.act = act;
    p.ctype = ytype;
    const bool vec = x.vec(K) && w.vec(K) && (groups == 1 || stride_w % 8 == 0);
    return status(launch_l16_fwd(type == LL_TYPE_BF16, p, vec, dev.cus, static_cast<hipStream_t>(stream)));
}

int64_t ll_linear16_grad_act_workspace_size(int M, int N, int groups)
{
    return M < 0 || N < 0 || groups < 0 || groups > LL_MAX_GROUPS ? -1 : 4 * act_grad_parts(M, N, groups);
}

int linear16_grad_act(int M, int N, int type, int act, int ytype, const void *DY, int lddy, int groups,
                      const int32_t *offsets, const uint16_t *Z, int ldz, const uint8_t *ZQ, int ldzq, const uint8_t *ZS,
                      int ldzs, uint16_t *DZ, int lddz, float *dbias, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!type16(type) || !out_type(ytype, type) || M < 0 || N < 0 || act < LL_ACT_NONE || act > LL_ACT_SILU ||
        !groups_ok(offsets, groups) || (ZQ == nullptr) != (ZS == nullptr) || (Z != nullptr && ZQ != nullptr) ||
        workspace_bytes < 0)
        return LL_ERR_INVALID_VALUE;
    const Mat dy{DY, lddy, type_bytes(ytype)}, z{Z, ldz, 2}, zq{ZQ, ldzq, 1}, zs{ZS, ldzs, 1}, dz{DZ, lddz, 2};
    const int nb = blocks_of(N);
    if (!dy.ld_ok(N) || !z.ld_ok(N) || !zq.ld_ok(N) || !zs.ld_ok(nb) || !dz.ld_ok(N))
        return LL_ERR_INVALID_VALUE;
    if (N == 0 || groups == 0 || (M == 0 && dbias == nullptr))
        return LL_OK;
    if (M > kL16Most || N > kL16Most || !aligned(dbias, 4) || (DZ == nullptr && dbias == nullptr))
        return LL_ERR_INVALID_VALUE;
    if (M > 0 && (DY == nullptr || (act != LL_ACT_NONE && Z == nullptr && ZQ == nullptr) || !dy.ok(M, N) || !z.ok(M, N) ||
                  !zq.ok(M, N) || !zs.ok(M, nb) || !dz.ok(M, N)))
        return LL_ERR_INVALID_VALUE;
    const int64_t need = dbias != nullptr ? 4 * act_grad_parts(M, N, groups) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
        return LL_ERR_INVALID_VALUE;
    // dz may be written over dy or z; nothing else may meet an output
    const Range out[3] = {vec_range(dbias, (int64_t)groups * N), {workspace, need}, dz.range(M, N)};
    const Range in[3] = {zq.range(M, N), zs.range(M, nb), groups_range(offsets, groups)};
    const Range dyr = dy.range(M, N), zr = z.range(M, N);
    if (any_overlap(out, 3, in, 3) || any_overlap(out, 2, &dyr, 1) || any_overlap(out, 2, &zr, 1) ||
        (!(dz.same(dy) && ytype == type) && overlap(out[2], dyr)) || (!dz.same(z) && overlap(out[2], zr)))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    const ActGradParams p{DY,  Z,    ZQ,   ZS,   DZ, dbias, dbias != nullptr ? static_cast<float *>(workspace) : nullptr,
                          lddy, ldz, ldzq, ldzs, lddz, Groups{offsets, groups}, M, N, act};
    return status(launch_act_grad(type == LL_TYPE_BF16, ytype, p, static_cast<hipStream_t>(stream)));
}

int linear16_grad_input(int M, int N, int K, int type, const uint16_t *DZ, int lddz, int groups, const int32_t *offsets,
                        const uint16_t *W, int ldw, int64_t stride_w, int xtype, void *DX, int lddx, void *workspace,
                        int64_t workspace_bytes, void *stream)
{
    if (workspace_bytes < 0 || !type16(type) || !out_type(xtype, type) || M < 0 || N < 0 || K < 0 || !groups_ok(offsets, groups) || stride_w < 0)
        return LL_ERR_INVALID_VALUE;
    const Mat dz{DZ, lddz, 2}, w{W, ldw, 2}, dx{DX, lddx, type_bytes(xtype)};
    if (!dz.ld_ok(N) || !w.ld_ok(K) || !dx.ld_ok(K))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || K == 0 || groups == 0)
        return LL_OK;
    const Range wr = stack_range(w, N, K, stride_w, groups);
    if (DX == nullptr || (N > 0 && (DZ == nullptr || W == nullptr)) || M > kL16Most || N > kL16Most || K > kL16Most ||
        !dz.ok(M, N) || !w.ok(N, K) || wr.bytes < 0 || !dx.ok(M, K))
        return LL_ERR_INVALID_VALUE;
    const Range out[1] = {dx.range(M, K)}, in[3] = {dz.range(M, N), wr, groups_range(offsets, groups)};
    if (any_overlap(out, 1, in, 3) || (workspace != nullptr && !aligned(workspace, 16)))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    const int shares = workspace != nullptr ? l16_shares(L16_DX, M, N, K, groups, dev.cus) : 1;
    const int64_t need = shares_bytes(shares, M, K);
    const Range ws = {workspace, need};
    if (need > 0 && (workspace_bytes < need || any_overlap(&ws, 1, in, 3) || overlap(ws, out[0])))
        return LL_ERR_INVALID_VALUE;
    L16Params p{};
    p.A = DZ;
    p.B = W;
    p.C = DX;
    p.lda = lddz, p.ldb = ldw, p.ldc = lddx;
    p.stride_b = stride_w;
    p.groups = Groups{offsets, groups};
    p.M = M, p.N = K, p.K = N;
    p.ctype = xtype;
    p.ws = static_cast<float *>(workspace);
    p.shares = shares;
    const bool vec = dz.vec(N) && w.vec(K) && (groups == 1 || stride_w % 8 == 0);
    return status(launch_l16_dx(type == LL_TYPE_BF16, p, vec, dev.cus, static_cast<hipStream_t>(stream)));
}

int linear16_grad_weight(int M, int N, int K, int type, const uint16_t *DZ, int lddz, int groups, const int32_t *offsets,
                         const uint16_t *X, int ldx, const uint8_t *XQ, int ldxq, const uint8_t *XS, int ldxs, int wtype,
                         float beta, void *DW, int lddw, int64_t stride_dw, void *stream)
{
    if (!type16(type) || !out_type(wtype, type) || M < 0 || N < 0 || K < 0 || !groups_ok(offsets, groups) ||
        (XQ == nullptr) != (XS == nullptr) || (X != nullptr && XQ != nullptr) || stride_dw < 0)
        return LL_ERR_INVALID_VALUE;
    const Mat dz{DZ, lddz, 2}, x{X, ldx, 2}, xq{XQ, ldxq, 1}, xs{XS, ldxs, 1}, dw{DW, lddw, type_bytes(wtype)};
    const int nb = blocks_of(K);
    if (!dz.ld_ok(N) || !x.ld_ok(K) || !xq.ld_ok(K) || !xs.ld_ok(nb) || !dw.ld_ok(K))
        return LL_ERR_INVALID_VALUE;
    if (N == 0 || K == 0 || groups == 0)
        return LL_OK;
    const Range dwr = stack_range(dw, N, K, stride_dw, groups);
    if (DW == nullptr || M > kL16Most || N > kL16Most || K > kL16Most || !dw.ok(N, K) || dwr.bytes < 0 ||
        (groups > 1 && stride_dw < (int64_t)(N - 1) * lddw + K))
        return LL_ERR_INVALID_VALUE;
    if (M > 0 && (DZ == nullptr || (X == nullptr && XQ == nullptr) || !dz.ok(M, N) || !x.ok(M, K) || !xq.ok(M, K) ||
                  !xs.ok(M, nb)))
        return LL_ERR_INVALID_VALUE;
    const Range in[5] = {dz.range(M, N), x.range(M, K), xq.range(M, K), xs.range(M, nb), groups_range(offsets, groups)};
    if (any_overlap(&dwr, 1, in, 5))
        return LL_ERR_INVALID_VALUE;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    L16Params p{};
    p.A = DZ;
    p.B = XQ != nullptr ? static_cast<const void *>(XQ) : X;
    p.BS = XS;
    p.C = DW;
    p.lda = lddz, p.ldb = XQ != nullptr ? ldxq : ldx, p.ldbs = ldxs, p.ldc = lddw;
    p.stride_c = stride_dw;
    p.groups = Groups{offsets, groups};
    p.M = N, p.N = K, p.K = M;
    p.shares = 1;
    p.ctype = wtype;
    p.beta = beta;
    // codes: rows on 16 bytes (the last piece may be short)
    const bool vec = dz.vec(N) && (XQ != nullptr ? aligned(XQ, 16) && ldxq % 16 == 0 && xq.ld < (int64_t)1 << 21 &&
                                                       ldxs < (int64_t)1 << 21
                                                 : x.vec(K));
    return status(launch_l16_dw(type == LL_TYPE_BF16, p, vec, dev.cus, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
