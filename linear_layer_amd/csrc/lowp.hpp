// Host-side launchers of the 4-bit format, its products and the residual norms.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ll {

hipError_t launch_mx4_quantize(int type, const void *X, int64_t ldx, bool trans, uint8_t *codes, int64_t ldq,
                               uint8_t *scales, int64_t lds, int M, int K, hipStream_t s);
hipError_t launch_mx4_dequantize(int type, const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                                 int64_t lds, void *Y, int64_t ldy, int M, int K, hipStream_t s);

// The first operand of a product: MX4 codes, or 16-bit values.
enum MxA : int { MXA_MX4 = 0, MXA_F16 = 1, MXA_BF16 = 2 };

// C = alpha * A * B^T + beta * C, B in MX4 (N rows of K), A in MX4 or 16 bits.
struct MxParams {
    const uint8_t *A;        // codes, or 16-bit values as bytes
    const uint8_t *SA;       // A's scales (MXA_MX4)
    const uint8_t *B, *SB;   // B's codes and scales
    float *C;
    int64_t lda, ldb;        // bytes between rows
    int64_t ldsa, ldsb;      // bytes between rows of scales
    int64_t ldc;             // elements
    int M, N, K;
    float alpha, beta;
    int tiles_m, tiles_n;
    int group_m;             // tile rows per group in the tiles' order
    int halved;              // tiles at its end done in two halves
    float *ws;               // room for the shares' sums, or null: K is not shared out
    int splits;              // shares of K
};

// Tiles of 256 x 256 or 128 x 128 (M and N at least that, K at least 512); `copies`:
// rows of 16-byte pieces, copied straight into LDS.
enum MxTile : int { MX_TILE_256 = 0, MX_TILE_128 = 1 };
hipError_t launch_gemm_mx4_tile(MxParams p, int a, int tile, bool copies, int cus, hipStream_t s);
// Bytes of workspace that make a product faster (0: none does).
int64_t mx4_workspace(int M, int N, int K, int a, int cus);
// The name of the kernel it takes.
const char *mx4_kernel_name(int M, int N, int K, int a, bool copies, bool workspace, int cus);
hipError_t launch_gemm_mx4(MxParams p, int a, int cus, hipStream_t s);

// The residual step between two blocks (rmsnorm.hip); null pointers leave parts out.
struct NormParams {
    const float *Y;                        // the block's output, or null
    const float *w_post, *gate, *w_pre;    // N values each, or null: ones
    const void *X;
    void *XO, *H;
    int64_t ldy, ldx, ldxo, ldh;           // elements
    int M, N;
    float alpha, eps;
};
hipError_t launch_rmsnorm_residual(int type, const NormParams &p, hipStream_t s);

struct NormGradParams {
    const float *Y, *w_post, *gate, *w_pre;
    const void *X, *DXO, *DH;
    float *DY;
    void *DX;
    float *DGATE, *DWPOST, *DWPRE;
    float *part;                           // partial column sums (set by the launcher)
    int64_t ldy, ldx, lddxo, lddh, lddy, lddx;
    int M, N;
    float alpha, eps;
    float eps_y;                           // eps of y's norm (set by the launcher)
};
// Bytes of the workspace launch_rmsnorm_grad uses.
int64_t rmsnorm_grad_workspace(int M, int N);
hipError_t launch_rmsnorm_grad(int type, NormGradParams p, void *ws, hipStream_t s);

}  // namespace ll
