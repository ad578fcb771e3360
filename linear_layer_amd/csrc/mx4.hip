// Quantisation to MX4 and back (see mx4.hpp for the format). Both directions
// are bound by HBM: a lane takes 8 values (16 or 32 bytes) and 4 bytes of
// codes, four neighbouring lanes make a block of 32. 8192 x 8192 bfloat16 there and
// back 67.6 us; each alone, through tensors past the cache, 35.8 (4.7 TB/s of values and
// codes; a large copy reaches 5.1 to 5.5) and 37.4, and along the columns 39.1 (4.4).
// 2047 x 11008 along the columns: FP32 24.8 us (4.1 TB/s), 16-bit types 24.0 (2.4: a row's
// 64 values are 128 bytes of them), against 20.7 and 14.4 along the rows.
#include "linear_layer.h"
#include "lowp.hpp"
#include "mx4.hpp"

namespace ll {

// Rows quantised along themselves. The (row, block, quarter) triples of a slab
// of rows are dealt out in order, so that short rows fill the lanes as well as
// long ones; a thread takes kQuantPer of them, a grid's stride apart, and has
// all their loads in flight together.
constexpr int kQuantPer = 4;

// The largest of v over groups of four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, false));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, false));
}

template <int TYPE>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const typename Elem<TYPE>::type *X, int64_t ldx,
                                                           uint8_t *codes, int64_t ldq, uint8_t *scales,
                                                           int64_t lds, uint32_t units, int K)
{
    const uint32_t upr = (uint32_t)((K - 1) / kMxBlock + 1) * 4u;   // lanes' units of a row
    const uint32_t step = gridDim.x * 256u, first = blockIdx.x * 256u + threadIdx.x;
    float v[kQuantPer][8];
    uint32_t row[kQuantPer], k[kQuantPer];
#pragma unroll
    for (int i = 0; i < kQuantPer; ++i) {
        const uint32_t u = first + i * step;
        row[i] = u / upr;
        k[i] = (u - row[i] * upr) * 8u;
        load_row<TYPE, 8>(X + (int64_t)row[i] * ldx + k[i], u < units ? (int64_t)K - k[i] : 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kQuantPer; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7fffffffu);
        const uint32_t s = mx_scale(quad_max(top)), c = mx_encode8(v[i], s);
        if (first + i * step >= units)
            continue;
        if ((threadIdx.x & 3) == 0)
            scales[(int64_t)row[i] * lds + k[i] / kMxBlock] = (uint8_t)s;
        uint8_t *dst = codes + (int64_t)row[i] * ldq + k[i] / 2;
        if ((int64_t)k[i] + 8 <= K) {
            __builtin_memcpy(dst, &c, 4);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((int64_t)k[i] + 2 * j < K)
                    dst[j] = (uint8_t)(c >> (8 * j));
        }
    }
}

// Columns quantised along themselves, written as the transposed matrix's rows.
// A workgroup takes 64 columns by 8 blocks of 32 rows. A lane reads the 32
// values of one column's block (each of the 32 loads is one row's 64
// neighbouring values, coalesced); the codes pass through LDS so that a
// transposed row gets its 8 blocks' 128 bytes in one piece (16-byte pieces at
// the transposed row stride would each touch a cache line of their own).
constexpr int kTransCols = 64, kTransBlocks = 8;

template <int TYPE>
__global__ void __launch_bounds__(64 * kTransBlocks)
mx4_quantize_trans_kernel(const typename Elem<TYPE>::type *X, int64_t ldx, uint8_t *codes, int64_t ldq,
                          uint8_t *scales, int64_t lds, int M, int K, int tiles_k)
{
    __shared__ u32x4 q[kTransCols][kTransBlocks + 1];   // one chunk more a row: spread over the banks
    __shared__ uint8_t sc[kTransCols][kTransBlocks];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tk = blockIdx.x % tiles_k, tm = blockIdx.x / tiles_k;
    const int64_t k0 = (int64_t)tk * kTransCols, m0 = ((int64_t)tm * kTransBlocks + wave) * kMxBlock;
    const int64_t k = k0 + lane;
    float v[kMxBlock];
    const typename Elem<TYPE>::type *src = X + m0 * ldx + k;
    if (k < K && m0 + kMxBlock <= M) {
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j)
            v[j] = to_f32<TYPE>(src[j * ldx]);
    } else {
#pragma unroll
        for (int j = 0; j < kMxBlock; ++j)
            v[j] = k < K && m0 + j < M ? to_f32<TYPE>(src[j * ldx]) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kMxBlock; ++j)
        top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7fffffffu);
    const uint32_t s = mx_scale(top);
    u32x4 c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        c[j] = mx_encode8(v + 8 * j, s);
    q[lane][wave] = c;
    sc[lane][wave] = (uint8_t)s;
    __syncthreads();
    // thread t: column t / 8's chunk t % 8
    const int col = threadIdx.x / kTransBlocks, b = threadIdx.x % kTransBlocks;
    const int64_t kk = k0 + col, m = ((int64_t)tm * kTransBlocks + b) * kMxBlock;
    if (kk >= K || m >= M)
        return;
    scales[kk * lds + m / kMxBlock] = sc[col][b];
    uint8_t *dst = codes + kk * ldq + m / 2;
    const u32x4 w = q[col][b];
    if (m + kMxBlock <= M) {
        __builtin_memcpy(dst, &w, 16);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (m + 2 * j < M)
                dst[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
}

// The values codes and scales stand for, rounded to TYPE (exact in FP32 and
// bfloat16 but for 6 * 2^127 and the like, which are infinite there; binary16
// rounds, and overflows past 65504).
template <int TYPE>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t *codes, int64_t ldq,
                                                             const uint8_t *scales, int64_t lds,
                                                             typename Elem<TYPE>::type *Y, int64_t ldy,
                                                             uint32_t units, int K)
{
    const uint32_t upr = (uint32_t)((K - 1) / kMxBlock + 1) * 4u;
    const uint32_t step = gridDim.x * 256u, first = blockIdx.x * 256u + threadIdx.x;
    uint32_t row[kQuantPer], k[kQuantPer], c[kQuantPer], s[kQuantPer];
#pragma unroll
    for (int i = 0; i < kQuantPer; ++i) {
        const uint32_t u = first + i * step;
        row[i] = u / upr;
        k[i] = (u - row[i] * upr) * 8u;
        c[i] = s[i] = 0;
        if (u < units && (int64_t)k[i] < K) {
            s[i] = scales[(int64_t)row[i] * lds + k[i] / kMxBlock];
            const uint8_t *src = codes + (int64_t)row[i] * ldq + k[i] / 2;
            if ((int64_t)k[i] + 8 <= K) {
                __builtin_memcpy(&c[i], src, 4);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((int64_t)k[i] + 2 * j < K)
                        c[i] |= (uint32_t)src[j] << (8 * j);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kQuantPer; ++i) {
        if (first + i * step >= units || (int64_t)k[i] >= K)
            continue;
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const float sc = __builtin_bit_cast(float, s[i] << 23);
        float v[8];
        const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 0);
        const f32x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 1);
        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 2);
        const f32x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 3);
        v[0] = p0[0], v[1] = p0[1], v[2] = p1[0], v[3] = p1[1];
        v[4] = p2[0], v[5] = p2[1], v[6] = p3[0], v[7] = p3[1];
        store_row<TYPE, 8>(Y + (int64_t)row[i] * ldy + k[i], (int64_t)K - k[i], v);
    }
}

// Rows of one launch, so that its units fit 31 bits.
static int slab_rows(int rows, int K)
{
    const int64_t most = ((int64_t)1 << 30) / (((int64_t)(K - 1) / kMxBlock + 1) * 4);
    return (int)(most < 1 ? 1 : most < rows ? most : rows);
}

static dim3 unit_grid(uint32_t units)
{
    return dim3((units + 256u * kQuantPer - 1) / (256u * kQuantPer));
}

template <int TYPE>
static hipError_t quantize_t(const void *X, int64_t ldx, bool trans, uint8_t *codes, int64_t ldq,
                             uint8_t *scales, int64_t lds, int M, int K, hipStream_t s)
{
    using T = typename Elem<TYPE>::type;
    const T *x = static_cast<const T *>(X);
    if (trans) {
        // launches of at most 2^30 work items: slabs of columns, and of rows of tiles
        constexpr int most = (1 << 30) / (64 * kTransBlocks), cols = most * kTransCols, tall = kTransBlocks * kMxBlock;
        const int tiles_m = cdiv(M, tall);
        for (int64_t k0 = 0; k0 < K; k0 += cols) {
            const int k = (int)(K - k0 < cols ? K - k0 : cols), tiles_k = cdiv(k, kTransCols), slab = most / tiles_k;
            for (int t = 0; t < tiles_m; t += slab) {
                const int n = tiles_m - t < slab ? tiles_m - t : slab;
                const int64_t m0 = (int64_t)t * tall;
                hipLaunchKernelGGL(mx4_quantize_trans_kernel<TYPE>, dim3((unsigned)(n * tiles_k)),
                                   dim3(64 * kTransBlocks), 0, s, x + m0 * ldx + k0, ldx, codes + k0 * ldq + m0 / 2, ldq,
                                   scales + k0 * lds + m0 / kMxBlock, lds, (int)(M - m0), k, tiles_k);
            }
        }
    } else {
        const int slab = slab_rows(M, K);
        for (int64_t m = 0; m < M; m += slab) {
            const int64_t n = M - m < slab ? M - m : slab;
            const uint32_t units = (uint32_t)(n * ((K - 1) / kMxBlock + 1) * 4);
            hipLaunchKernelGGL(mx4_quantize_kernel<TYPE>, unit_grid(units), dim3(256), 0, s, x + m * ldx,
                               ldx, codes + m * ldq, ldq, scales + m * lds, lds, units, K);
        }
    }
    return hipGetLastError();
}

hipError_t launch_mx4_quantize(int type, const void *X, int64_t ldx, bool trans, uint8_t *codes, int64_t ldq,
                               uint8_t *scales, int64_t lds, int M, int K, hipStream_t s)
{
    if (type == LL_TYPE_F32)
        return quantize_t<LL_TYPE_F32>(X, ldx, trans, codes, ldq, scales, lds, M, K, s);
    if (type == LL_TYPE_F16)
        return quantize_t<LL_TYPE_F16>(X, ldx, trans, codes, ldq, scales, lds, M, K, s);
    return quantize_t<LL_TYPE_BF16>(X, ldx, trans, codes, ldq, scales, lds, M, K, s);
}

template <int TYPE>
static hipError_t dequantize_t(const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                               void *Y, int64_t ldy, int M, int K, hipStream_t s)
{
    using T = typename Elem<TYPE>::type;
    const int slab = slab_rows(M, K);
    for (int64_t m = 0; m < M; m += slab) {
        const int64_t n = M - m < slab ? M - m : slab;
        const uint32_t units = (uint32_t)(n * ((K - 1) / kMxBlock + 1) * 4);
        hipLaunchKernelGGL(mx4_dequantize_kernel<TYPE>, unit_grid(units), dim3(256), 0, s, codes + m * ldq,
                           ldq, scales + m * lds, lds, static_cast<T *>(Y) + m * ldy, ldy, units, K);
    }
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(int type, const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                                 int64_t lds, void *Y, int64_t ldy, int M, int K, hipStream_t s)
{
    if (type == LL_TYPE_F32)
        return dequantize_t<LL_TYPE_F32>(codes, ldq, scales, lds, Y, ldy, M, K, s);
    if (type == LL_TYPE_F16)
        return dequantize_t<LL_TYPE_F16>(codes, ldq, scales, lds, Y, ldy, M, K, s);
    return dequantize_t<LL_TYPE_BF16>(codes, ldq, scales, lds, Y, ldy, M, K, s);
}

}  // namespace ll
