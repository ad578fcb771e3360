// The C ABI of the 4-bit microscaled format: argument checks, then one launch
// on the caller's stream. Nothing here allocates or synchronises.
#include <hip/hip_runtime.h>

#include "linear_layer.h"
#include "host.hpp"
#include "launch.hpp"
#include "lowp.hpp"

using namespace ll;
using namespace ll::host;

namespace {

// Bytes of a packed row of K codes, and its scales.
int64_t code_bytes(int K) { return ((int64_t)K + 1) / 2; }
int64_t scale_bytes(int K) { return ((int64_t)K + 31) / 32; }

int max1(int v) { return v > 1 ? v : 1; }

// A packed matrix of rows x K: leading dimensions, pointers, extents.
struct Packed {
    const void *codes, *scales;
    int rows, K, ldq, lds;
    bool lds_ok() const { return ldq >= max1((int)code_bytes(K)) && lds >= max1((int)scale_bytes(K)); }
    Range code_range() const { return {codes, span(rows, code_bytes(K), ldq, 1)}; }
    Range scale_range() const { return {scales, span(rows, scale_bytes(K), lds, 1)}; }
    bool ok() const
    {
        return codes != nullptr && scales != nullptr && code_range().bytes >= 0 && scale_range().bytes >= 0;
    }
};

// The form of A (LL_A_*) as the launchers name it.
bool known_form(int a) { return a == LL_A_MX4 || a == LL_A_F16 || a == LL_A_BF16; }
int form(int a) { return a == LL_A_MX4 ? MXA_MX4 : a == LL_A_F16 ? MXA_F16 : MXA_BF16; }

int quantize_args(int rows, int cols, int type, const void *X, int ldx, int x_rows, int x_cols, const Packed &q,
                  bool writes_x)
{
    const int es = type_bytes(type);
    if (es == 0 || rows < 0 || cols < 0 || ldx < max1(x_cols) || !q.lds_ok())
        return LL_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0)
        return LL_OK;
    const Range x{X, span(x_rows, x_cols, ldx, es)};
    if (X == nullptr || !aligned(X, es) || x.bytes < 0 || !q.ok())
        return LL_ERR_INVALID_VALUE;
    const Range packed[2] = {q.code_range(), q.scale_range()};
    if (writes_x ? any_overlap(&x, 1, packed, 2) : any_overlap(packed, 2, &x, 1))
        return LL_ERR_INVALID_VALUE;
    return LL_OK;
}

int gemm_mx4(int M, int N, int K, float alpha, int a, const void *A, int lda, const void *SA, int ldsa,
             const void *B, int ldb, const void *SB, int ldsb, float beta, float *C, int ldc, void *workspace,
             int64_t workspace_bytes, void *stream)
{
    if (M < 0 || N < 0 || K < 0 || ldc < max1(N) || workspace_bytes < 0)
        return LL_ERR_INVALID_VALUE;
    const Packed qa{A, SA, M, K, lda, ldsa}, qb{B, SB, N, K, ldb, ldsb};
    if (!qb.lds_ok() || (a == MXA_MX4 ? !qa.lds_ok() : lda < max1(K)))
        return LL_ERR_INVALID_VALUE;
    if (M == 0 || N == 0)
        return LL_OK;
    const Range c{C, span(M, N, ldc, 4)};
    if (C == nullptr || !aligned(C, 4) || c.bytes < 0)
        return LL_ERR_INVALID_VALUE;
    const bool product = K > 0 && alpha != 0.0f;
    if (product) {
        if (!qb.ok() || (a == MXA_MX4 ? !qa.ok() : A == nullptr || !aligned(A, 2)))
            return LL_ERR_INVALID_VALUE;
        const Range in[4] = {qb.code_range(), qb.scale_range(),
                             a == MXA_MX4 ? qa.code_range() : Range{A, span(M, K, lda, 2)},
                             a == MXA_MX4 ? qa.scale_range() : Range{nullptr, 0}};
        if (in[2].bytes < 0 || any_overlap(&c, 1, in, 4))
            return LL_ERR_INVALID_VALUE;
        const Range ws{workspace, workspace != nullptr ? workspace_bytes : 0};
        if (workspace != nullptr && (!aligned(workspace, 16) || any_overlap(&ws, 1, in, 4) || overlap(ws, c)))
            return LL_ERR_INVALID_VALUE;
    }
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!product)
        return status(launch_scale(C, ldc, M, N, beta, s));
    MxParams p;
    memset(&p, 0, sizeof p);
    p.A = static_cast<const uint8_t *>(A);
    p.SA = static_cast<const uint8_t *>(SA);
    p.B = static_cast<const uint8_t *>(B);
    p.SB = static_cast<const uint8_t *>(SB);
    p.C = C;
    p.lda = a == MXA_MX4 ? (int64_t)lda : (int64_t)lda * 2;
    p.ldb = ldb;
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.ldc = ldc;
    p.M = M;
    p.N = N;
    p.K = K;
    p.alpha = alpha;
    p.beta = beta;
    const int64_t need = workspace != nullptr ? mx4_workspace(M, N, K, a, dev.cus) : 0;
    if (need > 0) {
        if (workspace_bytes < need)
            return LL_ERR_INVALID_VALUE;
        p.ws = static_cast<float *>(workspace);
    }
    const hipError_t e = launch_gemm_mx4(p, a, dev.cus, s);
    return e == hipErrorInvalidValue ? LL_ERR_INVALID_VALUE : status(e);
}

}  // namespace

extern "C" {

int mx4_quantize(int M, int K, int type, const void *X, int ldx, int trans, uint8_t *codes, int ldq,
                 uint8_t *scales, int lds, void *stream)
{
    if (trans != 0 && trans != 1)
        return LL_ERR_INVALID_VALUE;
    const Packed q{codes, scales, trans ? K : M, trans ? M : K, ldq, lds};
    const int st = M < 0 || K < 0 ? LL_ERR_INVALID_VALUE : quantize_args(M, K, type, X, ldx, M, K, q, false);
    if (st != LL_OK || M == 0 || K == 0)
        return st;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    return status(launch_mx4_quantize(type, X, ldx, trans == 1, codes, ldq, scales, lds, M, K,
                                      static_cast<hipStream_t>(stream)));
}

int mx4_dequantize(int M, int K, const uint8_t *codes, int ldq, const uint8_t *scales, int lds, int type, void *Y,
                   int ldy, void *stream)
{
    const Packed q{codes, scales, M, K, ldq, lds};
    const int st = M < 0 || K < 0 ? LL_ERR_INVALID_VALUE : quantize_args(M, K, type, Y, ldy, M, K, q, true);
    if (st != LL_OK || M == 0 || K == 0)
        return st;
    const Device dev = current_device();
    if (dev.status != LL_OK)
        return dev.status;
    return status(launch_mx4_dequantize(type, codes, ldq, scales, lds, Y, ldy, M, K,
                                        static_cast<hipStream_t>(stream)));
}

int gemm_mx4f32_nt(int M, int N, int K, float alpha, const uint8_t *A, int lda, const uint8_t *SA, int ldsa,
                   const uint8_t *B, int ldb, const uint8_t *SB, int ldsb, float beta, float *C, int ldc,
                   void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_MX4, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C, ldc, nullptr, 0, stream);
}

int gemm_f16mx4f32_nt(int M, int N, int K, float alpha, const uint16_t *A, int lda, const uint8_t *B, int ldb,
                      const uint8_t *SB, int ldsb, float beta, float *C, int ldc, void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_F16, A, lda, nullptr, 0, B, ldb, SB, ldsb, beta, C, ldc, nullptr, 0, stream);
}

int gemm_bf16mx4f32_nt(int M, int N, int K, float alpha, const uint16_t *A, int lda, const uint8_t *B, int ldb,
                       const uint8_t *SB, int ldsb, float beta, float *C, int ldc, void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_BF16, A, lda, nullptr, 0, B, ldb, SB, ldsb, beta, C, ldc, nullptr, 0, stream);
}

int64_t ll_mx4_workspace_size(int M, int N, int K, int a)
{
    if (M < 0 || N < 0 || K < 0 || !known_form(a))
        return -1;
    const Device dev = current_device();
    return mx4_workspace(M, N, K, form(a), dev.status == LL_OK ? dev.cus : 256);
}

const char *ll_mx4_chosen_kernel(int M, int N, int K, int a, int aligned, int workspace, int num_cus)
{
    return known_form(a) ? mx4_kernel_name(M, N, K, form(a), aligned != 0, workspace != 0, num_cus > 0 ? num_cus : 256) : "";
}

int gemm_mx4f32_nt_ws(int M, int N, int K, float alpha, const uint8_t *A, int lda, const uint8_t *SA, int ldsa,
                      const uint8_t *B, int ldb, const uint8_t *SB, int ldsb, float beta, float *C, int ldc,
                      void *workspace, int64_t workspace_bytes, void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_MX4, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C, ldc, workspace, workspace_bytes,
                    stream);
}

int gemm_f16mx4f32_nt_ws(int M, int N, int K, float alpha, const uint16_t *A, int lda, const uint8_t *B, int ldb,
                         const uint8_t *SB, int ldsb, float beta, float *C, int ldc, void *workspace,
                         int64_t workspace_bytes, void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_F16, A, lda, nullptr, 0, B, ldb, SB, ldsb, beta, C, ldc, workspace, workspace_bytes,
                    stream);
}

int gemm_bf16mx4f32_nt_ws(int M, int N, int K, float alpha, const uint16_t *A, int lda, const uint8_t *B, int ldb,
                          const uint8_t *SB, int ldsb, float beta, float *C, int ldc, void *workspace,
                          int64_t workspace_bytes, void *stream)
{
    return gemm_mx4(M, N, K, alpha, MXA_BF16, A, lda, nullptr, 0, B, ldb, SB, ldsb, beta, C, ldc, workspace, workspace_bytes,
                    stream);
}

}  // extern "C"
