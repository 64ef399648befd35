// Microscaled 4-bit floating point, to and fro: blocks of 32 elements along the inner
// axis share a power of two, the elements are E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a
// sign).  The shared exponent is that of the block's largest value less 2, so that
// value comes to 4 .. 8 and what passes 6 is clipped there (the OCP microscaling
// format's conversion); rounding to nearest, ties to even, by the hardware's
// conversion, which divides by the power of two exactly.
//
// All of it is bound by memory: 2 bytes in, 0.53 out (bf16).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "mxfp4.h"

namespace mamba {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kExpNan = 255;

// The scale's code (exponent + 127) of a block whose largest |x| has these fp32 bits:
// as unsigned integers |x| are in the order of their values, infinity and NaN on top.
__device__ __forceinline__ uint32_t scale_code(uint32_t top)
{
    const uint32_t e = top >> 23;
    return e == kExpNan ? kExpNan : (e > 2 ? e - 2 : 0);
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    const uint32_t o = __builtin_amdgcn_mov_dpp(v, 0xB1, 0xF, 0xF, true);
    v = v > o ? v : o;
    const uint32_t p = __builtin_amdgcn_mov_dpp(v, 0x4E, 0xF, 0xF, true);
    return v > p ? v : p;
}

// Eight values in 4 bits each, the first lowest.  The conversion reads its scale's
// exponent field, so code 0 (2^-127) needs no denormal.
__device__ __forceinline__ uint32_t pack8(const float (&f)[8], uint32_t code)
{
    if (code == kExpNan)
        return 0;
    const float s = __uint_as_float(code << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], s, 3);
    return w;
}

// ---- token-major ---------------------------------------------------------------------
// A workgroup takes ROWS rows of one group: 32 lanes a row, 8 elements a lane, so four
// lanes a block.  Scales go out by way of LDS, ROWS * 8 bytes in one piece.
template <int ROWS, bool BF16> __global__ __launch_bounds__(256) void quantize_kernel(const MxQuantArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kUnits = ROWS / 8;
    __shared__ uint32_t codes[ROWS * kMxScales / 4];
    const int64_t groups = mx_groups(p.K), rows = p.B * p.L;
    const int64_t g = blockIdx.x % groups, row0 = blockIdx.x / groups * ROWS;
    const int lane = threadIdx.x & 31;
    const int64_t k = g * kMxGroup + lane * 8;
    float f[kUnits][8];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t row = row0 + u * 8 + threadIdx.x / 32;
        const T *x = (const T *)p.x + row * p.K + k;
        if (row < rows && k + 8 <= p.K) {
            if constexpr (BF16) {
                u32x4 v;
                __builtin_memcpy(&v, x, 16);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[u][j] = __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
            } else {
                __builtin_memcpy(f[u], x, 32);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[u][j] = row < rows && k + j < p.K ? Elem<BF16>::load(x + j) : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int in = u * 8 + threadIdx.x / 32;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(f[u][j]) & 0x7fffffffu;
            top = top > b ? top : b;
        }
        const uint32_t code = scale_code(quad_max(top));
        const uint32_t w = pack8(f[u], code);
        if (row0 + in < rows)
            *(uint32_t *)(p.q + ((row0 + in) * groups + g) * kMxGroupBytes + lane * 4) = w;
        if ((lane & 3) == 0)
            ((uint8_t *)codes)[in * kMxScales + lane / 4] = (uint8_t)code;
    }
    __syncthreads();
    if (threadIdx.x < ROWS * 2 && row0 + threadIdx.x / 2 < rows)
        *(uint32_t *)(p.scale + (g * rows + row0) * kMxScales + threadIdx.x * 4) = codes[threadIdx.x];
}

// ---- channel-major ---------------------------------------------------------------------
// x [B, K, L] to rows (b, t) of K.  A workgroup takes one group of channels and 64
// tokens; a wave takes one block of 32 channels, a lane a token, so that its loads run
// along the tokens and a block's largest value needs no other lane.
template <bool BF16> __global__ __launch_bounds__(512) void quantize_channel_kernel(const MxQuantArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kTokens = 64;
    const int64_t groups = mx_groups(p.K), rows = p.B * p.L, tiles = (p.L + kTokens - 1) / kTokens;
    const int64_t tile = blockIdx.x % tiles, g = blockIdx.x / tiles % groups, b = blockIdx.x / tiles / groups;
    const int lane = threadIdx.x & 63, block = threadIdx.x / 64;
    const int64_t t = tile * kTokens + lane, k = g * kMxGroup + block * 32;
    if (t >= p.L)
        return;
    const T *x = (const T *)p.x + (b * p.K + k) * p.L + t;
    float f[4][8];
#pragma unroll
    for (int j = 0; j < 32; ++j)
        f[j / 8][j % 8] = k + j < p.K ? Elem<BF16>::load(x + (int64_t)j * p.L) : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const uint32_t v = __float_as_uint(f[j / 8][j % 8]) & 0x7fffffffu;
        top = top > v ? top : v;
    }
    const uint32_t code = scale_code(top);
    const u32x4 w = {pack8(f[0], code), pack8(f[1], code), pack8(f[2], code), pack8(f[3], code)};
    const int64_t row = b * p.L + t;
    *(u32x4 *)(p.q + (row * groups + g) * kMxGroupBytes + block * 16) = w;
    p.scale[(g * rows + row) * kMxScales + block] = (uint8_t)code;
}

// ---- back ------------------------------------------------------------------------------
// A lane takes 8 elements; the product with the power of two is exact but where it
// leaves the range of fp32.
template <bool BF16> __global__ __launch_bounds__(256) void dequantize_kernel(const MxDequantArgs p)
{
    using T = typename Elem<BF16>::T;
    const int64_t groups = mx_groups(p.K);
    const int64_t g = blockIdx.x % groups, row = blockIdx.x / groups * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    const int64_t k = g * kMxGroup + lane * 8;
    if (row >= p.rows || k >= p.K)
        return;
    const uint32_t w = *(const uint32_t *)(p.q + (row * groups + g) * kMxGroupBytes + lane * 4);
    const uint32_t code = p.scale[(g * p.rows + row) * kMxScales + lane / 4];
    const float s = __uint_as_float(code == kExpNan ? 0x7fc00000u : (code ? code << 23 : 0x00400000u));
    float f[8];
    typedef float f32x2v __attribute__((ext_vector_type(2)));
    const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1),
                 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
    f[0] = a[0] * s, f[1] = a[1] * s, f[2] = b[0] * s, f[3] = b[1] * s;
    f[4] = c[0] * s, f[5] = c[1] * s, f[6] = d[0] * s, f[7] = d[1] * s;
    T *o = (T *)p.out + row * p.K + k;
    if (k + 8 <= p.K) {
        if constexpr (BF16) {
            const u32x4 v = {cvt2(f[0], f[1]), cvt2(f[2], f[3]), cvt2(f[4], f[5]), cvt2(f[6], f[7])};
            __builtin_memcpy(o, &v, 16);
        } else {
            __builtin_memcpy(o, f, 32);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (k + j < p.K)
                Elem<BF16>::store(o + j, f[j]);
    }
}

}  // namespace

hipError_t launch_quantize_mxfp4(const MxQuantArgs &a, hipStream_t s)
{
    const int64_t rows = a.B * a.L, groups = mx_groups(a.K);
    const bool few = rows * groups < 32 * 1024;
    const dim3 grid((unsigned)(few ? (rows + 7) / 8 * groups : (rows + 31) / 32 * groups)), block(256);
    if (a.bf16 && few)
        quantize_kernel<8, true><<<grid, block, 0, s>>>(a);
    else if (a.bf16)
        quantize_kernel<32, true><<<grid, block, 0, s>>>(a);
    else if (few)
        quantize_kernel<8, false><<<grid, block, 0, s>>>(a);
    else
        quantize_kernel<32, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_quantize_mxfp4_channel_major(const MxQuantArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.L + 63) / 64 * mx_groups(a.K) * a.B)), block(512);
    if (a.bf16)
        quantize_channel_kernel<true><<<grid, block, 0, s>>>(a);
    else
        quantize_channel_kernel<false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const MxDequantArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.rows + 7) / 8 * mx_groups(a.K))), block(256);
    if (a.bf16)
        dequantize_kernel<true><<<grid, block, 0, s>>>(a);
    else
        dequantize_kernel<false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mamba
