// Microscaled 8-bit floating point, there and back, and the gradient of the layer's
// activation, which can read its input from it. All are bound by HBM: a lane takes 8 values
// (16 or 32 bytes, 8 of codes), four neighbouring lanes make a block of 32. 8192 x 8192 bfloat16
// there and back: 82 us for 338 MB (4.1 TB/s); the gradient with its sums of 8191 x 4096, SiLU: 47 us
// for 169 MB (3.6 TB/s).
#include "linear16.hpp"
#include "launch.hpp"

namespace ll {

// The (row, block, quarter) triples of a slab of rows are dealt out in order, so that short
// rows fill the lanes as well as long ones; a thread takes kPer of them, a grid's stride
// apart, and has all their loads in flight together.
constexpr int kPer = 4;

template <int TYPE>
__global__ void __launch_bounds__(256) mx8_quantize_kernel(const typename Elem<TYPE>::type *X, int64_t ldx, uint8_t *codes,
                                                           int64_t ldq, uint8_t *scales, int64_t lds, uint32_t units, int K)
{
    const uint32_t upr = (uint32_t)((K - 1) / kMxBlock + 1) * 4u;   // lanes' units of a row
    const uint32_t step = gridDim.x * 256u, first = blockIdx.x * 256u + threadIdx.x;
    float v[kPer][8];
    uint32_t row[kPer], k[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t u = first + i * step;
        row[i] = u / upr;
        k[i] = (u - row[i] * upr) * 8u;
        load_row<TYPE, 8>(X + (int64_t)row[i] * ldx + k[i], u < units ? (int64_t)K - k[i] : 0, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            top = max(top, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7fffffffu);
        const uint32_t s = mx8_scale(max_of_quad(top));
        if (first + i * step >= units || (int64_t)k[i] >= K)
            continue;
        const uint64_t q = (uint64_t)mx8_encode4(v[i][4], v[i][5], v[i][6], v[i][7], s) << 32 |
                           mx8_encode4(v[i][0], v[i][1], v[i][2], v[i][3], s);
        if ((threadIdx.x & 3) == 0)
            scales[(int64_t)row[i] * lds + k[i] / kMxBlock] = (uint8_t)s;
        uint8_t *dst = codes + (int64_t)row[i] * ldq + k[i];
        if ((int64_t)k[i] + 8 <= K) {
            __builtin_memcpy(dst, &q, 8);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((int64_t)k[i] + j < K)
                    dst[j] = (uint8_t)(q >> (8 * j));
        }
    }
}

// Eight codes of a row from `src` on, the first n of them inside it.
__device__ __forceinline__ uint64_t load_codes(const uint8_t *src, int64_t n)
{
    uint64_t c = 0;
    if (n >= 8) {
        __builtin_memcpy(&c, src, 8);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n)
                c |= (uint64_t)src[j] << (8 * j);
    }
    return c;
}

template <int TYPE>
__global__ void __launch_bounds__(256) mx8_dequantize_kernel(const uint8_t *codes, int64_t ldq, const uint8_t *scales,
                                                             int64_t lds, typename Elem<TYPE>::type *Y, int64_t ldy,
                                                             uint32_t units, int K)
{
    const uint32_t upr = (uint32_t)((K - 1) / kMxBlock + 1) * 4u;
    const uint32_t step = gridDim.x * 256u, first = blockIdx.x * 256u + threadIdx.x;
    uint32_t row[kPer], k[kPer], s[kPer];
    uint64_t c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t u = first + i * step;
        row[i] = u / upr;
        k[i] = (u - row[i] * upr) * 8u;
        c[i] = s[i] = 0;
        if (u < units && (int64_t)k[i] < K) {
            s[i] = scales[(int64_t)row[i] * lds + k[i] / kMxBlock];
            c[i] = load_codes(codes + (int64_t)row[i] * ldq + k[i], (int64_t)K - k[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (first + i * step >= units || (int64_t)k[i] >= K)
            continue;
        float v[8];
        mx8_decode4((uint32_t)c[i], s[i], v);
        mx8_decode4((uint32_t)(c[i] >> 32), s[i], v + 4);
        store_row<TYPE, 8>(Y + (int64_t)row[i] * ldy + k[i], (int64_t)K - k[i], v);
    }
}

// Rows of one launch, so that its units fit 31 bits.
static int slab_rows(int rows, int K)
{
    const int64_t most = ((int64_t)1 << 30) / (((int64_t)(K - 1) / kMxBlock + 1) * 4);
    return (int)(most < 1 ? 1 : most < rows ? most : rows);
}

static dim3 unit_grid(uint32_t units) { return dim3((units + 256u * kPer - 1) / (256u * kPer)); }

template <int TYPE>
static hipError_t quantize_t(const void *X, int64_t ldx, uint8_t *codes, int64_t ldq, uint8_t *scales, int64_t lds, int M,
                             int K, hipStream_t s)
{
    const auto *x = static_cast<const typename Elem<TYPE>::type *>(X);
    const int slab = slab_rows(M, K);
    for (int64_t m = 0; m < M; m += slab) {
        const int64_t n = M - m < slab ? M - m : slab;
        const uint32_t units = (uint32_t)(n * ((K - 1) / kMxBlock + 1) * 4);
        hipLaunchKernelGGL(mx8_quantize_kernel<TYPE>, unit_grid(units), dim3(256), 0, s, x + m * ldx, ldx, codes + m * ldq,
                           ldq, scales + m * lds, lds, units, K);
    }
    return hipGetLastError();
}

hipError_t launch_mx8_quantize(int type, const void *X, int64_t ldx, uint8_t *codes, int64_t ldq, uint8_t *scales,
                               int64_t lds, int M, int K, hipStream_t s)
{
    if (type == LL_TYPE_F32)
        return quantize_t<LL_TYPE_F32>(X, ldx, codes, ldq, scales, lds, M, K, s);
    if (type == LL_TYPE_F16)
        return quantize_t<LL_TYPE_F16>(X, ldx, codes, ldq, scales, lds, M, K, s);
    return quantize_t<LL_TYPE_BF16>(X, ldx, codes, ldq, scales, lds, M, K, s);
}

template <int TYPE>
static hipError_t dequantize_t(const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds, void *Y, int64_t ldy,
                               int M, int K, hipStream_t s)
{
    auto *y = static_cast<typename Elem<TYPE>::type *>(Y);
    const int slab = slab_rows(M, K);
    for (int64_t m = 0; m < M; m += slab) {
        const int64_t n = M - m < slab ? M - m : slab;
        const uint32_t units = (uint32_t)(n * ((K - 1) / kMxBlock + 1) * 4);
        hipLaunchKernelGGL(mx8_dequantize_kernel<TYPE>, unit_grid(units), dim3(256), 0, s, codes + m * ldq, ldq,
                           scales + m * lds, lds, y + m * ldy, ldy, units, K);
    }
    return hipGetLastError();
}

hipError_t launch_mx8_dequantize(int type, const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                                 void *Y, int64_t ldy, int M, int K, hipStream_t s)
{
    if (type == LL_TYPE_F32)
        return dequantize_t<LL_TYPE_F32>(codes, ldq, scales, lds, Y, ldy, M, K, s);
    if (type == LL_TYPE_F16)
        return dequantize_t<LL_TYPE_F16>(codes, ldq, scales, lds, Y, ldy, M, K, s);
    return dequantize_t<LL_TYPE_BF16>(codes, ldq, scales, lds, Y, ldy, M, K, s);
}

// ---- the activation's gradient -----------------------------------------------------

// dZ = dY * act'(Z), and the sums of dZ over each group's rows. A workgroup takes a chunk of
// rows of one group by a strip of 8 * lpr columns (lpr lanes a row, a power of two from 8 to 64),
// its 256 / lpr rows at a time from kActRows loads of each in flight; its column sums go to
// `part`, a row for every chunk, and a second launch adds a group's chunks in order. (Atomics
// would add them in any order.) Two rows in flight a thread and five waves a SIMD: 8191 x 4096 with Z
// in 8 bits 47 us with the second launch (3.6 TB/s); four rows and three waves 71.
constexpr int kActRows = 2;

// Rows of a chunk: 64 (the partial sums then are 1/32 of dZ's bytes); 16 where that leaves CUs
// without work. With 16 and with 64, SiLU, Z in 8 bits: 1000 x 4096 12.4 and 22.4 us, 1024 x 4096 12.7 and 22.5,
// 2048 x 4096 13.7 and 22.8, 8192 x 4096 46.4 and 43.3, 65536 x 128 (one group's 4096 chunks to join) 30.9 and
// 15.3: the border suits long columns and is low for wide rows.
static int act_step(int M, int N) { return (int64_t)M * N >= ((int64_t)1 << 22) ? 64 : 16; }

static int64_t act_chunks(int M, int N, int groups)
{
    return (int64_t)M / act_step(M, N) + (groups < M ? groups : M);
}

int64_t act_grad_parts(int M, int N, int groups) { return act_chunks(M, N, groups) * N; }

enum ZForm : int { Z_NONE = 0, Z_16 = 1, Z_8 = 2 };

template <bool BF16, int DYT, int ZF>
__global__ void __launch_bounds__(256) act_grad_kernel(ActGradParams p, int step, int lpr, int strips)
{
    constexpr int T = BF16 ? LL_TYPE_BF16 : LL_TYPE_F16;
    __shared__ float red[256][9];   // (9: the sums' reads spread over the banks)
    Chunk c;
    const int id = blockIdx.x / strips;
    if (id >= find_chunk(p.groups, p.M, step, id, c))
        return;
    const int tid = threadIdx.x, rows = 256 / lpr;
    const int64_t col = (int64_t)(blockIdx.x % strips) * lpr * 8 + tid % lpr * 8;
    const int64_t n = (int64_t)p.N - col;
    const int64_t r0 = (int64_t)c.begin + (int64_t)c.index * step, r1 = min(r0 + step, (int64_t)c.end);
    float sum[8] = {};
    for (int64_t r = r0 + tid / lpr; r < r1; r += (int64_t)rows * kActRows) {
        float dy[kActRows][8], z[kActRows][8];
        uint64_t codes[kActRows];
        uint32_t scale[kActRows];
#pragma unroll
        for (int i = 0; i < kActRows; ++i) {
            const int64_t m = r + i * rows, live = m < r1 ? n : 0;
            load_row<DYT, 8>(static_cast<const typename Elem<DYT>::type *>(p.DY) + m * p.lddy + col, live, dy[i]);
            if constexpr (ZF == Z_16) {
                load_row<T, 8>(p.Z + m * p.ldz + col, live, z[i]);
            } else if constexpr (ZF == Z_8) {
                codes[i] = load_codes(p.ZQ + m * p.ldzq + col, live);
                scale[i] = live > 0 ? p.ZS[m * p.ldzs + col / kMxBlock] : 0;
            }
        }
        if constexpr (ZF == Z_8) {
#pragma unroll
            for (int i = 0; i < kActRows; ++i) {
                mx8_decode4((uint32_t)codes[i], scale[i], z[i]);
                mx8_decode4((uint32_t)(codes[i] >> 32), scale[i], z[i] + 4);
            }
        }
        if constexpr (ZF != Z_NONE)   // (the sums are FP32, dZ is not)
            with_activation(act_for(p.act, p.part != nullptr), [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < kActRows; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dy[i][e] *= activation_slope<decltype(kind)::value>(z[i][e]);
            });
#pragma unroll
        for (int i = 0; i < kActRows; ++i) {
            const int64_t m = r + i * rows;
            if (m >= r1 || n <= 0)
                continue;
            if (p.DZ != nullptr)
                store_row<T, 8>(p.DZ + m * p.lddz + col, n, dy[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += dy[i][e];
        }
    }
    if (p.part == nullptr)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        red[tid][e] = sum[e];
    __syncthreads();
    for (int k = tid; k < lpr * 8; k += 256) {
        float t = 0.0f;
        for (int r = 0; r < rows; ++r)
            t += red[r * lpr + k / 8][k % 8];
        const int64_t at = (int64_t)(blockIdx.x % strips) * lpr * 8 + k;
        if (at < p.N)
            p.part[(int64_t)id * p.N + at] = t;
    }
}

// A group's chunks added up: 64 columns by SHARES of the chunks, then the shares in order. (Of 16
// groups of 8191 rows, 9 chunks each, with 16 shares 51.0 us in all, with 4 46.8.)
template <int SHARES>
__global__ void __launch_bounds__(64 * SHARES) act_join_kernel(const float *part, float *dbias, Groups groups, int M,
                                                                    int N, int step, int strips)
{
    __shared__ float red[SHARES][64];
    Chunk c{0, 0, 0, 0, 0};
    const int g = blockIdx.x / strips;
    find_chunk<true>(groups, M, step, g, c);
    const int64_t col = (int64_t)(blockIdx.x % strips) * 64 + threadIdx.x % 64;
    const int share = threadIdx.x / 64;
    float sum = 0.0f;
    if (col < N) {
#pragma unroll 8
        for (int i = share; i < c.index; i += SHARES)
            sum += part[(int64_t)(c.group_first + i) * N + col];
    }
    red[share][threadIdx.x % 64] = sum;
    __syncthreads();
    if (share == 0 && col < N) {
#pragma unroll
        for (int i = 1; i < SHARES; ++i)
            sum += red[i][threadIdx.x];
        dbias[(int64_t)g * N + col] = sum;
    }
}

template <bool BF16, int DYT>
static hipError_t launch_act_grad_t(const ActGradParams &p, hipStream_t s)
{
    int lpr = 8;
    while (lpr < 64 && lpr * 8 < p.N)
        lpr *= 2;
    const int step = act_step(p.M, p.N), strips = cdiv(p.N, lpr * 8);
    const int64_t chunks = p.groups.offsets == nullptr ? cdiv(p.M, step) : act_chunks(p.M, p.N, p.groups.n);
    const int64_t grid = chunks * strips;
    if (grid > max_grid_x(256) || (int64_t)p.groups.n * cdiv(p.N, 64) > max_grid_x(1024))
        return hipErrorInvalidValue;
    if (grid > 0) {
        const dim3 d((unsigned)grid);
        if (p.act == LL_ACT_NONE)
            hipLaunchKernelGGL((act_grad_kernel<BF16, DYT, Z_NONE>), d, dim3(256), 0, s, p, step, lpr, strips);
        else if (p.Z != nullptr)
            hipLaunchKernelGGL((act_grad_kernel<BF16, DYT, Z_16>), d, dim3(256), 0, s, p, step, lpr, strips);
        else
            hipLaunchKernelGGL((act_grad_kernel<BF16, DYT, Z_8>), d, dim3(256), 0, s, p, step, lpr, strips);
    }
    if (p.dbias != nullptr) {
        const dim3 d((unsigned)(p.groups.n * cdiv(p.N, 64)));
        if (chunks > (int64_t)16 * p.groups.n)
            hipLaunchKernelGGL(act_join_kernel<16>, d, dim3(1024), 0, s, p.part, p.dbias, p.groups, p.M, p.N, step, cdiv(p.N, 64));
        else
            hipLaunchKernelGGL(act_join_kernel<4>, d, dim3(256), 0, s, p.part, p.dbias, p.groups, p.M, p.N, step, cdiv(p.N, 64));
    }
    return hipGetLastError();
}

hipError_t launch_act_grad(bool bf16, int dytype, ActGradParams p, hipStream_t s)
{
    if (dytype == LL_TYPE_F32)
        return bf16 ? launch_act_grad_t<true, LL_TYPE_F32>(p, s) : launch_act_grad_t<false, LL_TYPE_F32>(p, s);
    return bf16 ? launch_act_grad_t<true, LL_TYPE_BF16>(p, s) : launch_act_grad_t<false, LL_TYPE_F16>(p, s);
}

}  // namespace ll
