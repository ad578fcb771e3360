// The 16-bit layer (linear16_nt), its gradients and the 8-bit format they can
// read and write: parameter blocks, host-side launchers, and the device code
// that the kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "common.hpp"
#include "linear_layer.h"
#include "mx4.hpp"

namespace ll {

// Rows that belong together (one expert's): group g has the rows from offsets[g]
// on, up to offsets[g + 1]. offsets == nullptr: one group of all rows.
struct Groups {
    const int32_t *offsets;
    int n;
};

// One product. Forward: C (M x N) = A (M x K) * W_g^T (N x K) with its write-back.
// Input gradient: C (M x N) = A (M x K) * W_g (K x N). Weight gradient: C_g (M x N) =
// A^T * B over the rows of group g, A (K rows in all x M), B (K rows x N).
struct L16Params {
    const uint16_t *A;
    const void *B;              // 16-bit values, or E4M3 codes
    const uint8_t *BS;          // B's scales
    void *C;
    const float *bias;          // groups x N, or null
    const void *R;              // added after the activation, of C's type, or null
    uint16_t *Z;                // A * W^T + bias in A's type, or null
    uint8_t *ZQ, *ZS;           // the same in 8 bits, or null
    float *ws;                  // room for the shares' sums
    int64_t lda, ldb, ldc, ldr, ldz;        // elements
    int64_t ldbs, ldzq, ldzs;               // bytes
    int64_t stride_b, stride_c;             // elements between groups' weights
    Groups groups;
    int M, N, K;
    int act;
    int ctype;                  // LL_TYPE_* of C (and R)
    float beta;
    int tiles_n, tiles_m;       // set by the launcher
    int shares;                 // of K (or of the rows), summed through ws
};

enum L16Op : int { L16_FWD = 0, L16_DX = 1, L16_DW = 2 };

// `vec`: every row of 16-bit operands in whole 16-byte pieces, on 16 bytes.
hipError_t launch_l16_fwd(bool bf16, L16Params p, bool vec, int cus, hipStream_t s);
// The forward product of few rows a group, and in how many shares of K it gains from a
// workspace.
bool l16_takes_rows(int M, int groups);
int l16_row_shares(int M, int N, int K, int groups, int cus);
// In how many shares of the contracted axis a product (op: forward or input gradient; M rows, N
// outputs, K inputs of the layer) gains from a workspace of that many times its result in FP32.
int l16_shares(int op, int M, int N, int K, int groups, int cus);
// The shares added in order, and the write-back (after a product in p.shares > 1).
hipError_t launch_l16_join(bool bf16, const L16Params &p, hipStream_t s);
hipError_t launch_l16_rows(bool bf16, const L16Params &p, bool vec, int cus, hipStream_t s);
hipError_t launch_l16_dx(bool bf16, L16Params p, bool vec, int cus, hipStream_t s);
hipError_t launch_l16_dw(bool bf16, L16Params p, bool vec, int cus, hipStream_t s);

// The name of the kernel that one of them takes: M rows, N outputs and K inputs of the layer.
const char *l16_kernel_name(int op, int M, int N, int K, int groups, bool vec, int cus);

struct ActGradParams {
    const void *DY;             // M x N of LL_TYPE_*
    const uint16_t *Z;          // 16 bits, or
    const uint8_t *ZQ, *ZS;     // 8 bits, or neither
    uint16_t *DZ;               // or null
    float *dbias;               // groups x N, or null
    float *part;                // partial column sums
    int64_t lddy, ldz, ldzq, ldzs, lddz;
    Groups groups;
    int M, N;
    int act;
};
// Floats of `part`.
int64_t act_grad_parts(int M, int N, int groups);
// Most sums, rows and columns that one call may have (their numbers, and those a tile past
// them, are 32-bit).
constexpr int kL16Most = 0x7fffffff - 1024;
hipError_t launch_act_grad(bool bf16, int dytype, ActGradParams p, hipStream_t s);

hipError_t launch_mx8_quantize(int type, const void *X, int64_t ldx, uint8_t *codes, int64_t ldq, uint8_t *scales,
                               int64_t lds, int M, int K, hipStream_t s);
hipError_t launch_mx8_dequantize(int type, const uint8_t *codes, int64_t ldq, const uint8_t *scales, int64_t lds,
                                 void *Y, int64_t ldy, int M, int K, hipStream_t s);

// ---- groups of rows ------------------------------------------------------------

// Where a group begins, whatever stands in `offsets`: values are taken into 0 .. M
// and a group never begins before the one ahead of it, so wrong offsets give wrong
// rows but no access outside the matrices and no row in two groups.
__device__ __forceinline__ int wave_max_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d)
            v = max(v, o);
    }
    return v;
}

__device__ __forceinline__ int wave_sum_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d)
            v += o;
    }
    return v;
}

// The rows [begin, end) of group g. Every lane of the wave takes part.
__device__ __forceinline__ void group_rows(const Groups &gr, int M, int g, int &begin, int &end)
{
    if (gr.offsets == nullptr) {
        begin = 0;
        end = M;
        return;
    }
    const int lane = threadIdx.x & 63;
    int top = 0;
    for (int i = lane; i <= g; i += 64)
        top = max(top, gr.offsets[i]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        top = max(top, __shfl_xor(top, d));
    begin = min(max(top, 0), M);
    end = min(max(top, gr.offsets[g + 1]), M);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(max(begin, end));
}

// Rows of all groups cut into chunks of at most `step`, group by group. Returns their
// number; c: chunk `id` (its group, the group's rows, its number within the group and the
// id of the group's first chunk), or with BY_GROUP those of group `id` (index: how many
// chunks it has). An id that is no chunk's leaves c alone. Every lane of the wave takes part.
struct Chunk {
    int group, begin, end, index, group_first;
};
// find_chunk_by: a group of r rows has count(r) of them, in whatever form.
template <bool BY_GROUP = false, class Count>
__device__ __forceinline__ int find_chunk_by(const Groups &gr, int M, Count count, int id, Chunk &c)
{
    if (gr.offsets == nullptr) {
        c = Chunk{0, 0, M, BY_GROUP ? count(M) : id, 0};
        return count(M);
    }
    const int lane = threadIdx.x & 63;
    int top = min(max(gr.offsets[0], 0), M), chunks = 0;
    for (int g0 = 0; g0 < gr.n; g0 += 64) {
        const int g = g0 + lane;
        int e = g < gr.n ? min(max(gr.offsets[g + 1], 0), M) : 0;
        e = max(wave_max_scan(e), top);
        const int before = __shfl_up(e, 1);
        const int b = lane == 0 ? top : before;
        const int n = g < gr.n ? count(e - b) : 0;
        const int incl = wave_sum_scan(n) + chunks, excl = incl - n;
        const unsigned long long hit = __ballot(BY_GROUP ? g == id : id >= excl && id < incl);
        if (hit != 0) {
            const int src = __ffsll(hit) - 1, first = __shfl(excl, src);
            c = Chunk{g0 + src, __shfl(b, src), __shfl(e, src), BY_GROUP ? __shfl(n, src) : id - first, first};
        }
        top = __shfl(e, 63);
        chunks = __shfl(incl, 63);
    }
    c.group = __builtin_amdgcn_readfirstlane(c.group);
    c.begin = __builtin_amdgcn_readfirstlane(c.begin);
    c.end = __builtin_amdgcn_readfirstlane(c.end);
    c.index = __builtin_amdgcn_readfirstlane(c.index);
    c.group_first = __builtin_amdgcn_readfirstlane(c.group_first);
    return __builtin_amdgcn_readfirstlane(chunks);
}
template <bool BY_GROUP = false>
__device__ __forceinline__ int find_chunk(const Groups &gr, int M, int step, int id, Chunk &c)
{
    return find_chunk_by<BY_GROUP>(gr, M, [step](int rows) { return cdiv(rows, step); }, id, c);
}

// ---- activations ----------------------------------------------------------------

constexpr float kGeluA = 0.7978845608028654f;     // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + exp(-v)). The reciprocal and the exponential are the hardware's (one unit in the
// last place): a full division takes ten instructions, and a tile's write-back has a wave to itself.
__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// The normal distribution function at z, and e = exp(-z^2 / 2), for results of 16 bits. For x = |z| /
// sqrt(2) and t = 1 / (1 + p x), erfc(x) is a polynomial of t times exp(-x^2) to 1.5e-7 (Abramowitz
// and Stegun, Handbook of Mathematical Functions, 7.1.26). The bound is absolute: relative to the
// value the polynomial is off by 5e-5 at z = -3, 2e-3 at -5, where GELU is -1.4e-6, and 1e-2 at -8.
__device__ __forceinline__ float normal_cdf16(float z, float &e)
{
    const float x = __builtin_fabsf(z) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
    float q = __builtin_fmaf(1.061405429f, t, -1.453152027f);
    q = __builtin_fmaf(q, t, 1.421413741f);
    q = __builtin_fmaf(q, t, -0.284496736f);
    q = __builtin_fmaf(q, t, 0.254829592f);
    e = __builtin_amdgcn_exp2f(x * x * -1.4426950408889634f);
    const float h = 0.5f * q * t * e;
    return z > 0.0f ? 1.0f - h : h;
}

// The same for results of 32 bits, good relative to its value. Inside (-1, 1) it is 1/2 + z P(z^2),
// P to 7e-10; outside, on the negative side, exp(-z^2 / 2) t Q(t) with t = 1 / (1 + 0.4 |z|), t Q(t)
// to 8e-8 up to |z| = 13.5. (Minimax fits of P and Q to the function in 64 bits.) GELU of normal values
// is off by 3.7e-8 in the norm, as 0.5 z (1 + erf(z / sqrt(2))) in FP32 is; by the polynomial above 9e-8,
// which a result of 16 bits does not show and is nine operations less: 2047 x 11008 x 4096 to FP32 173 us
// with that and 180 with this, to bfloat16 170 and 178; the gradient with sums of 8191 x 4096 50 and 55.
__device__ __forceinline__ float normal_cdf32(float z, float &e)
{
    const float u = z * z, x = __builtin_fabsf(z);
    float c = __builtin_fmaf(-7.656804e-06f, u, 0.000113493545f);
    c = __builtin_fmaf(c, u, -0.0011863372f);
    c = __builtin_fmaf(c, u, 0.009973327f);
    c = __builtin_fmaf(c, u, -0.06649036f);
    c = __builtin_fmaf(c, u, 0.3989423f);
    c = __builtin_fmaf(c, z, 0.5f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f, x, 1.0f));
    float q = __builtin_fmaf(0.06812132f, t, -0.18642788f);
    q = __builtin_fmaf(q, t, 0.10536302f);
    q = __builtin_fmaf(q, t, 0.055540644f);
    q = __builtin_fmaf(q, t, 0.13900228f);
    q = __builtin_fmaf(q, t, 0.1591f);
    q = __builtin_fmaf(q, t, 0.15959579f);
    e = __builtin_amdgcn_exp2f(u * -0.72134752044448170f);
    const float h = q * t * e, f = z > 0.0f ? 1.0f - h : h;
    return x < 1.0f ? c : f;
}

// z times a factor that goes to 0 as z goes to minus infinity.
__device__ __forceinline__ float damped(float z, float f) { return f == 0.0f ? 0.0f : z * f; }

// GELU with normal_cdf32, beside the LL_ACT_*, and the kind that results of FP32 (or not) take.
constexpr int kActGelu32 = LL_ACT_SILU + 1;
constexpr int act_for(int act, bool f32) { return act == LL_ACT_GELU && f32 ? kActGelu32 : act; }

// act(z). The tanh form of GELU is z * sigmoid(2 u): 0.5 * (1 + tanh(u)) is that.
template <int ACT>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == LL_ACT_RELU) {
        return z > 0.0f ? z : 0.0f;
    } else if constexpr (ACT == LL_ACT_GELU) {
        float e;
        return damped(z, normal_cdf16(z, e));
    } else if constexpr (ACT == kActGelu32) {
        float e;
        return damped(z, normal_cdf32(z, e));
    } else if constexpr (ACT == LL_ACT_GELU_TANH) {
        return damped(z, sigmoid(2.0f * kGeluA * __builtin_fmaf(kGeluB * z * z, z, z)));
    } else if constexpr (ACT == LL_ACT_SILU) {
        return damped(z, sigmoid(z));
    } else {
        return z;
    }
}

// act'(z). Past +-110 every slope here is 0 or 1 in FP32 to the last bit; as a factor z is held
// there, so that no product of an infinity and a zero comes up (NaN stays NaN through the other).
template <int ACT>
__device__ __forceinline__ float activation_slope(float z)
{
    const float f = __builtin_amdgcn_fmed3f(z, -110.0f, 110.0f);
    if constexpr (ACT == LL_ACT_RELU) {
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == LL_ACT_GELU || ACT == kActGelu32) {
        float e;
        const float c = ACT == kActGelu32 ? normal_cdf32(z, e) : normal_cdf16(z, e);
        return __builtin_fmaf(f * 0.3989422804014327f, e, c);
    } else if constexpr (ACT == LL_ACT_GELU_TANH) {
        const float s = sigmoid(2.0f * kGeluA * __builtin_fmaf(kGeluB * z * z, z, z));
        return __builtin_fmaf(f * s * (1.0f - s), 2.0f * kGeluA * __builtin_fmaf(3.0f * kGeluB * f, f, 1.0f), s);
    } else if constexpr (ACT == LL_ACT_SILU) {
        const float s = sigmoid(z);
        return __builtin_fmaf(f * s, 1.0f - s, s);
    } else {
        return 1.0f;
    }
}

// f(std::integral_constant<int, act>): one test of the kind for all that f does with it.
template <class F>
__device__ __forceinline__ void with_activation(int act, F f)
{
    switch (act) {
    case LL_ACT_RELU: f(std::integral_constant<int, LL_ACT_RELU>{}); break;
    case LL_ACT_GELU: f(std::integral_constant<int, LL_ACT_GELU>{}); break;
    case LL_ACT_GELU_TANH: f(std::integral_constant<int, LL_ACT_GELU_TANH>{}); break;
    case LL_ACT_SILU: f(std::integral_constant<int, LL_ACT_SILU>{}); break;
    case kActGelu32: f(std::integral_constant<int, kActGelu32>{}); break;
    default: f(std::integral_constant<int, LL_ACT_NONE>{}); break;
    }
}

// ---- 8-bit values -----------------------------------------------------------------

// The scale byte of a block whose largest magnitude has the FP32 pattern `top`:
// 127 + e with e the smallest exponent, at least -127, for which the magnitude is at
// most 448 * 2^e (E4M3's largest value), so that nothing is clipped; 255 for a block with
// an infinity or a NaN. 448 is 1.75 * 2^8: past that fraction the exponent is one more. A
// subnormal magnitude gives 0.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t top)
{
    const uint32_t e = top >> 23;
    if (e == 255u)
        return 255u;
    const uint32_t up = e + ((top & 0x7fffffu) > 0x600000u ? 1u : 0u);
    return up > 8u ? up - 8u : 0u;
}

// Four E4M3 codes of four values under scale byte s (< 255), to nearest, ties to
// even. The conversion takes the scale from an FP32 value's exponent field (0: 2^-127).
__device__ __forceinline__ uint32_t mx8_encode4(float v0, float v1, float v2, float v3, uint32_t s)
{
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float sc = __builtin_bit_cast(float, s << 23);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v0, v1, sc, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v2, v3, sc, true);
    return s == 255u ? 0u : __builtin_bit_cast(uint32_t, r);
}

// The values of four codes under scale byte s (255: NaN, which the conversion makes of its
// infinite scale).
__device__ __forceinline__ void mx8_decode4(uint32_t c, uint32_t s, float *v)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const float sc = __builtin_bit_cast(float, s << 23);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, sc, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, sc, true);
    v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1];
}

// The same in 16 bits, two a word, as a factor of a product: what rounding to 8 bits carried past
// binary16's range (65504 becomes 65536, under a scale of 2^8 or more) is its largest value.
template <bool BF16>
__device__ __forceinline__ void mx8_decode4(uint32_t c, uint32_t s, uint32_t &w0, uint32_t &w1)
{
    const float sc = __builtin_bit_cast(float, s << 23);
    if constexpr (BF16) {
        w0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, false));
        w1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, sc, true));
    } else {
        w0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, sc, false));
        w1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, sc, true));
        if (s >= 135u) {
            const auto held = [](uint32_t w) {
                w = (w & 0x7fffu) == 0x7c00u ? w - 1u : w;
                return (w & 0x7fff0000u) == 0x7c000000u ? w - 0x10000u : w;
            };
            w0 = held(w0);
            w1 = held(w1);
        }
    }
}

// The largest of v over groups of four lanes.
__device__ __forceinline__ uint32_t max_of_quad(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, false));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, false));
}

}  // namespace ll
