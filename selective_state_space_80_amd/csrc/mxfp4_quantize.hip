// Microscaled 4-bit floating point, to and fro: blocks of 32 elements along the inner
// axis share a power of two, the elements are E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a
// sign).  The shared exponent is that of the block's largest value less 2, so that
// value comes to 4 .. 8 and what passes 6 is clipped there (the OCP microscaling
// format's conversion); rounding to nearest, ties to even, by the hardware's
// conversion, which divides by the power of two exactly.
//
// All of it is bound by memory: 2 bytes in, 0.53 out (bf16).  8 x 5120 x 2048, inputs
// from memory: bf16 token-major 39.5 us, channel-major 38.0 (5.6 TB/s; a large copy moves
// 5.1 to 5.4), fp32 67.8 and 75.3, back to bf16 31, to fp32 55.
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
    const uint32_t n_groups = (uint32_t)groups, g = blockIdx.x % n_groups;  // blocks are below 2^24
    const int64_t row0 = (int64_t)(blockIdx.x / n_groups) * ROWS;
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
// x [B, K, L] to rows (b, t) of K.  A workgroup takes one group of channels and 128
// tokens (bf16; 64 in fp32); a wave takes one block of 32 channels, a lane two tokens
// (one), so that a load instruction takes 256 bytes of a channel and a block's largest
// value needs no other lane.  The packed rows go out by way of LDS, whole lines of 128
// bytes (chunk c of token t at c ^ (t / 2 % 8)), and so do the scales.
template <bool BF16> __global__ __launch_bounds__(512) void quantize_channel_kernel(const MxQuantArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kEach = BF16 ? 2 : 1, kTokens = 64 * kEach;
    __shared__ __attribute__((aligned(16))) uint8_t rows_out[kTokens * kMxGroupBytes];
    __shared__ __attribute__((aligned(16))) uint8_t scales_out[kTokens * kMxScales];
    const int64_t groups = mx_groups(p.K), rows = p.B * p.L, tiles = (p.L + kTokens - 1) / kTokens;
    const uint32_t n_tiles = (uint32_t)tiles, n_groups = (uint32_t)groups;  // blocks are below 2^23
    const int64_t tile = blockIdx.x % n_tiles, g = blockIdx.x / n_tiles % n_groups, b = blockIdx.x / n_tiles / n_groups;
    const int lane = threadIdx.x & 63, block = threadIdx.x / 64;
    const int64_t t = tile * kTokens + lane * kEach, k = g * kMxGroup + block * 32;
    const int left = p.K - k < 32 ? (p.K > k ? (int)(p.K - k) : 0) : 32;  // channels of this block
    const T *x = (const T *)p.x + (b * p.K + k) * p.L + t;
    uint32_t v[32];  // a channel each; bf16: two tokens, the first in the low half
    if (t + kEach <= p.L) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            v[j] = 0;
            if (j < left)
                __builtin_memcpy(&v[j], x + (int64_t)j * p.L, 4);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[j] = BF16 && t < p.L && j < left ? (uint32_t)x[(int64_t)j * p.L] : 0;
    }
    auto put = [&](int token, uint32_t code, u32x4 w) {
        *(u32x4 *)(rows_out + token * kMxGroupBytes + (block ^ ((token >> 1) & 7)) * 16) = w;
        scales_out[token * kMxScales + block] = (uint8_t)code;
    };
    if constexpr (BF16) {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 top = {0, 0};  // without their signs, bf16 are in the order of their bits
#pragma unroll
        for (int j = 0; j < 32; ++j)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[j] & 0x7fff7fffu));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t code = scale_code((uint32_t)top[h] << 16);
            const float s = __uint_as_float(code << 23);
            u32x4 w = {0, 0, 0, 0};
            auto pair = [&](int j) {  // this token's channels j and j + 1
                return __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(v[j + 1], v[j], h ? 0x07060302u : 0x05040100u));
            };
            if (code != kExpNan) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t q = 0;
                    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(c * 8), s, 0);
                    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(c * 8 + 2), s, 1);
                    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(c * 8 + 4), s, 2);
                    w[c] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, pair(c * 8 + 6), s, 3);
                }
            }
            put(lane * 2 + h, code, w);
        }
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j)
            top = top > (v[j] & 0x7fffffffu) ? top : v[j] & 0x7fffffffu;
        const uint32_t code = scale_code(top);
        u32x4 w;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = __uint_as_float(v[c * 8 + j]);
            w[c] = pack8(f, code);
        }
        put(lane, code, w);
    }
    __syncthreads();
    const int64_t row0 = b * p.L + tile * kTokens;
    const int tokens = p.L - tile * kTokens < kTokens ? (int)(p.L - tile * kTokens) : kTokens;
#pragma unroll
    for (int i = 0; i < kTokens / 64; ++i) {
        const int token = i * 64 + threadIdx.x / 8, c = threadIdx.x & 7;
        if (token < tokens)
            *(u32x4 *)(p.q + ((row0 + token) * groups + g) * kMxGroupBytes + c * 16) =
                *(const u32x4 *)(rows_out + token * kMxGroupBytes + (c ^ ((token >> 1) & 7)) * 16);
    }
    if (threadIdx.x < tokens)
        *(u32x2 *)(p.scale + (g * rows + row0 + threadIdx.x) * kMxScales) =
            *(const u32x2 *)(scales_out + threadIdx.x * kMxScales);
}

// ---- back ------------------------------------------------------------------------------
// A lane takes what it stores in 16 bytes, 8 elements (bf16) or 4, so that a wave's store
// is one piece, of several rows, and stores it past the caches (8 x 2048 x 5120 in fp32:
// 55 us; by the caches 102, with 8 elements a lane and two half-empty stores 123; bf16
// 31).  The product with the power of two is exact but where it leaves the type's range.
template <int ROWS, bool BF16> __global__ __launch_bounds__(256) void dequantize_kernel(const MxDequantArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kEach = BF16 ? 8 : 4, kLanes = kMxGroup / kEach, kPass = 256 / kLanes, kUnits = ROWS / kPass;
    const int64_t groups = mx_groups(p.K);
    const uint32_t n_groups = (uint32_t)groups, g = blockIdx.x % n_groups;
    const int64_t row0 = (int64_t)(blockIdx.x / n_groups) * ROWS + threadIdx.x / kLanes;
    const int lane = threadIdx.x & (kLanes - 1);
    const int64_t k = g * kMxGroup + lane * kEach;
    if (k >= p.K)
        return;
    uint32_t w[kUnits], codes[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t row = row0 + u * kPass < p.rows ? row0 + u * kPass : p.rows - 1;
        const uint8_t *q = p.q + (row * groups + g) * kMxGroupBytes + lane * kEach / 2;
        w[u] = BF16 ? *(const uint32_t *)q : *(const uint16_t *)q;
        codes[u] = p.scale[(g * p.rows + row) * kMxScales + lane * kEach / 32];
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int64_t row = row0 + u * kPass;
        if (row >= p.rows)
            return;
        const uint32_t code = codes[u];
        const float s = __uint_as_float(code == kExpNan ? 0x7fc00000u : (code ? code << 23 : 0x00400000u));
        typedef float f32x2v __attribute__((ext_vector_type(2)));
        f32x2v v[kEach / 2];
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.f, 0);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.f, 1);
        if constexpr (BF16) {
            v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.f, 2);
            v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.f, 3);
        }
        float f[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j)
            f[j] = v[j / 2][j % 2] * s;
        T *o = (T *)p.out + row * p.K + k;
        if (k + kEach <= p.K) {
            if constexpr (BF16) {
                const u32x4 b = {cvt2(f[0], f[1]), cvt2(f[2], f[3]), cvt2(f[4], f[5]), cvt2(f[6], f[7])};
                typedef u32x4 __attribute__((aligned(2))) loose;
                __builtin_nontemporal_store(b, (loose *)o);
            } else {
                typedef f32x4 __attribute__((aligned(4))) loose;
                __builtin_nontemporal_store(f32x4{f[0], f[1], f[2], f[3]}, (loose *)o);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kEach - 1; ++j)
                if (k + j < p.K)
                    Elem<BF16>::store(o + j, f[j]);
        }
    }
}

}  // namespace

// Units of 8 rows and a group: four a workgroup, whose loads are in flight together,
// where that still leaves work for every CU.
static bool four_units(int64_t rows, int64_t groups) { return rows * groups >= 32 * 1024; }

hipError_t launch_quantize_mxfp4(const MxQuantArgs &a, hipStream_t s)
{
    const int64_t rows = a.B * a.L, groups = mx_groups(a.K);
    const bool four = four_units(rows, groups);
    const dim3 grid((unsigned)(four ? (rows + 31) / 32 * groups : (rows + 7) / 8 * groups)), block(256);
    if (a.bf16 && four)
        quantize_kernel<32, true><<<grid, block, 0, s>>>(a);
    else if (a.bf16)
        quantize_kernel<8, true><<<grid, block, 0, s>>>(a);
    else if (four)
        quantize_kernel<32, false><<<grid, block, 0, s>>>(a);
    else
        quantize_kernel<8, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_quantize_mxfp4_channel_major(const MxQuantArgs &a, hipStream_t s)
{
    const int64_t tokens = a.bf16 ? 128 : 64;
    const dim3 grid((unsigned)((a.L + tokens - 1) / tokens * mx_groups(a.K) * a.B)), block(512);
    if (a.bf16)
        quantize_channel_kernel<true><<<grid, block, 0, s>>>(a);
    else
        quantize_channel_kernel<false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_dequantize_mxfp4(const MxDequantArgs &a, hipStream_t s)
{
    const int64_t groups = mx_groups(a.K);
    const bool four = four_units(a.rows, groups);
    const dim3 grid((unsigned)(four ? (a.rows + 31) / 32 * groups : (a.rows + 7) / 8 * groups)), block(256);
    if (a.bf16 && four)
        dequantize_kernel<32, true><<<grid, block, 0, s>>>(a);
    else if (a.bf16)
        dequantize_kernel<8, true><<<grid, block, 0, s>>>(a);
    else if (four)
        dequantize_kernel<32, false><<<grid, block, 0, s>>>(a);
    else
        dequantize_kernel<8, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mamba
