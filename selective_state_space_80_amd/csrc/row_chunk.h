// Device helpers of the row operators (norms, quantiser): a row of D elements
// in the registers of its lanes, 8-element chunks, sums and largest values
// over a wave, and the 8-bit rounding.
#pragma once

#include <hip/hip_runtime.h>

#include "device_common.h"

namespace mamba {
namespace {

constexpr int kChunk = 8;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 elements at any element's alignment (rows of odd width start at any
// element; gfx950 loads and stores 16 bytes at any address).
template <bool BF16> __device__ __forceinline__ void load8(const typename Elem<BF16>::T *p, float (&v)[8])
{
    if constexpr (BF16) {
        u32x4 r;
        __builtin_memcpy(&r, p, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
        }
    } else {
        u32x4 r0, r1;
        __builtin_memcpy(&r0, p, 16);
        __builtin_memcpy(&r1, p + 4, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(r0[i]);
            v[4 + i] = __uint_as_float(r1[i]);
        }
    }
}

template <bool BF16> __device__ __forceinline__ void store8(typename Elem<BF16>::T *p, const float (&v)[8])
{
    if constexpr (BF16) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = cvt2(v[2 * i], v[2 * i + 1]);
        __builtin_memcpy(p, &r, 16);
    } else {
        u32x4 r0, r1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r0[i] = __float_as_uint(v[i]);
            r1[i] = __float_as_uint(v[4 + i]);
        }
        __builtin_memcpy(p, &r0, 16);
        __builtin_memcpy(p + 4, &r1, 16);
    }
}

template <int CTRL> __device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL> __device__ __forceinline__ float dppf(float v)
{
    return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}

// Sum / unsigned maximum over each LANES (8, 16, 32 or 64) neighbouring lanes,
// in every one of them: quads, half rows, rows of 16 by DPP, then rows by a
// lane exchange, or of the whole wave through scalar registers.  A fixed order.
template <int LANES> __device__ __forceinline__ float lane_sum(float v)
{
    v = quad_sum(v);
    v += dppf<0x141>(v);  // row_half_mirror
    if constexpr (LANES >= 16)
        v += dppf<0x140>(v);  // row_mirror
    if constexpr (LANES == 32)
        v += __shfl_xor(v, 16);
    if constexpr (LANES < 64)
        return v;
    const int b = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) +
            __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(b, 32)) +
            __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int LANES> __device__ __forceinline__ uint32_t lane_max(uint32_t v)
{
    v = umax(v, dpp<0xB1>(v));
    v = umax(v, dpp<0x4E>(v));
    v = umax(v, dpp<0x141>(v));
    if constexpr (LANES >= 16)
        v = umax(v, dpp<0x140>(v));
    if constexpr (LANES == 32)
        v = umax(v, (uint32_t)__shfl_xor((int)v, 16));
    if constexpr (LANES < 64)
        return v;
    const int b = (int)v;
    return umax(umax((uint32_t)__builtin_amdgcn_readlane(b, 0), (uint32_t)__builtin_amdgcn_readlane(b, 16)),
                umax((uint32_t)__builtin_amdgcn_readlane(b, 32), (uint32_t)__builtin_amdgcn_readlane(b, 48)));
}

// Factor to take a row's elements by where the sum of their squares, s, leaves
// the fp32 range; the square sum and eps are then formed again with it.
//   s infinite: 2^-80.  The largest element is above 2^56, its square above 2^-48
//     then, and 32768 times the largest square there is is below 2^111.
//   s and eps below 2^-80: 2^100.  Elements are below 2^-40, the smallest number
//     there is becomes 2^-49.  (With s above 2^-80 what underflows in it is below
//     2^-54 of it; with eps above, s matters to 2^-54 of eps at most.)
__device__ __forceinline__ float range_factor(float s, float eps)
{
    if (s == __builtin_inff())
        return 0x1p-80f;
    return s < 0x1p-80f && eps < 0x1p-80f ? 0x1p100f : 1.f;
}

// 1 / sqrt(x) rounded once, for a normal x: the hardware's, off by up to a unit in
// the last place, and one step r + r (1 - x r^2) / 2 of which no part is rounded
// before it is small.  (The reciprocal of a rounded root rounds twice: up to 0.75
// units from 1 / sqrt(x) where this is 0.5.)  0 and NaN of infinity and NaN, as
// 1 / sqrt; x is normal or one of these, since small sums are taken by a power of
// two.
__device__ __forceinline__ float inv_root(float x)
{
    const float r = __builtin_amdgcn_rsqf(x);
    const float t = x * r, low = fmaf(x, r, -t);  // x r = t + low
    const float e = fmaf(-low, r, fmaf(-t, r, 1.f));
    return x < __builtin_inff() ? fmaf(0.5f * r, e, r) : r;
}

// Lanes that share a row of D elements where a wave holds whole rows: as few
// as hold it in one chunk each (8 rows of 64 elements a wave), 64 for longer.
inline int row_lanes(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// The bits of |v| order as |v| does, infinity above every finite value and NaN
// above infinity, so one unsigned maximum also tells a row that is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// q = the integer nearest to v * 127 / top, ties to even, in [-127, 127], for a
// row whose largest |value| is top.  Adding 1.5 * 2^23 to an fp32 number (2^52 in
// fp64) rounds it to an integer, whose low byte is then that integer in two's
// complement.  127 / top is no fp32 or fp64 number, so the product with its
// rounded value can miss a tie.  A first rounding to a fixed fraction, coarser
// than the miss but finer than the distance of any other quotient from a tie,
// puts it back:
//   bf16 values: v / top = a / (b 2^s) with integers a, b < 256.  A quotient that
//     is no tie is at least 1 / (b 2^s) > 1.54e-5 from one (254 a and odd
//     multiples of b 2^s are even for s > 0; for s = 0, 1 / 2b).  The fp32 product
//     misses by at most 127 * 2^-24 = 0.76e-5; rounded to multiples of 2^-15,
//     numbers within 1.53e-5 of a tie become it.
//   fp32 values: a, b < 2^24, the distance is at least 2^-33; the fp64 product
//     misses by at most 2^-38, and is rounded to multiples of 2^-36.
// One more instruction than a single rounding in bf16, two more for fp32 values
// (8 x 5120 x 2048 channel-major: bf16 69.4 us, 68.9 with the single rounding;
// fp32 104.8, 103.4; 131072 rows of 64, the norm's fp32 values, 7.6 and 7.1).
//
// A zero row has scale 0; a row that is not finite has scale NaN and q = 0, so
// that everything computed from it is NaN.
template <bool BF16> struct RowScale;
template <> struct RowScale<true> {
    float scale, mul;
    float raise;  // below 2^-120 the multiplier would pass the fp32 range: such rows are raised by 2^64
    uint32_t mask;
    __device__ __forceinline__ RowScale() = default;
    __device__ __forceinline__ explicit RowScale(uint32_t top)
    {
        const bool finite = top < 0x7f800000u;
        const float t = __uint_as_float(top);
        raise = top != 0 && t < 0x1p-120f ? 0x1p64f : 1.f;
        scale = finite ? t / 127.f : __uint_as_float(0x7fc00000u);
        mul = top == 0 || !finite ? 0.f : 127.f / (t * raise);
        mask = finite ? 0xffffffffu : 0u;
    }
    __device__ __forceinline__ uint32_t nearest(float v) const
    {
        constexpr float kFraction = 384.f, kInteger = 12582912.f;  // 1.5 * 2^8, 2^23
        return __float_as_uint(fmaf(v, mul, kFraction) + (kInteger - kFraction));
    }
};
template <> struct RowScale<false> {
    static constexpr float raise = 1.f;  // fp64 has room
    double mul;
    float scale;
    uint32_t mask;
    __device__ __forceinline__ RowScale() = default;
    __device__ __forceinline__ explicit RowScale(uint32_t top)
    {
        const bool finite = top < 0x7f800000u;
        const float t = __uint_as_float(top);
        scale = finite ? t / 127.f : __uint_as_float(0x7fc00000u);
        const float up = t < 0x1p-64f ? 0x1p64f : 1.f;
        const double m = (double)(127.f / (t * up)) * (double)up;  // the fp32 quotient, and its remainder's: 46 bits
        mul = top == 0 || !finite ? 0. : fma(fma(-m, (double)t, 127.), m * (1. / 127.), m);
        mask = finite ? 0xffffffffu : 0u;
    }
    __device__ __forceinline__ uint32_t nearest(float v) const
    {
        constexpr double kFraction = 0x1.8p16, kInteger = 0x1.8p52;
        return (uint32_t)__double_as_longlong(fma((double)v, mul, kFraction) + (kInteger - kFraction));
    }
};

// Bytes of four integers.
__device__ __forceinline__ uint32_t pack4(const uint32_t *b)
{
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
template <bool BF16> __device__ __forceinline__ u32x2 pack_int8(const float (&v)[8], const RowScale<BF16> &row)
{
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i] = row.nearest(v[i]);
    return u32x2{pack4(b), pack4(b + 4)} & row.mask;
}

// Where a lane's chunk of 8 elements lies in a row of D, and which of them are
// its own.  A row that is no multiple of 8 ends in a chunk that is moved back
// to end with the row: it overlaps the one before, computes the same values
// there, and owns only the elements from `lo` on.  Rows shorter than a chunk
// (TINY) are read element by element with the index held below D.
struct ChunkAt {
    int off, lo;
    bool live;
};
template <bool TINY> __device__ __forceinline__ ChunkAt chunk_at(int c, int D)
{
    const int full = D / kChunk, tail = D % kChunk;
    ChunkAt r;
    if (TINY) {
        r.off = 0;
        r.lo = 0;
        r.live = c == 0;
    } else {
        const bool last = tail != 0 && c == full;
        r.off = c < full ? c * kChunk : (last ? D - kChunk : 0);
        r.lo = last ? kChunk - tail : 0;
        r.live = c < full || last;
    }
    return r;
}

template <bool BF16, bool TINY>
__device__ __forceinline__ void load_chunk(const typename Elem<BF16>::T *row, const ChunkAt &at, int D,
                                           float (&v)[8])
{
    if constexpr (TINY) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = Elem<BF16>::load(row + (i < D ? i : D - 1));
    } else {
        load8<BF16>(row + at.off, v);
    }
}
// A chunk as it lies in memory, to be unpacked later.
template <bool BF16> struct RawChunk {
    u32x4 v[BF16 ? 1 : 2];
    template <bool TINY>
    __device__ __forceinline__ void load(const typename Elem<BF16>::T *row, const ChunkAt &at, int D)
    {
        if constexpr (TINY) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const typename Elem<BF16>::T e = row[i < D ? i : D - 1];
                if constexpr (BF16)
                    v[0][i / 2] = i % 2 ? v[0][i / 2] | (uint32_t)e << 16 : (uint32_t)e;
                else
                    v[i / 4][i % 4] = __float_as_uint(e);
            }
        } else {
#pragma unroll
            for (int i = 0; i < (BF16 ? 1 : 2); ++i)
                __builtin_memcpy(&v[i], row + at.off + 4 * i, 16);
        }
    }
    __device__ __forceinline__ void keep()
    {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            asm volatile("" : "+v"(v[i]));
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (BF16)
                f[i] = __uint_as_float(i % 2 ? v[0][i / 2] & 0xffff0000u : v[0][i / 2] << 16);
            else
                f[i] = __uint_as_float(v[i / 4][i % 4]);
        }
    }
};
template <bool BF16, bool TINY>
__device__ __forceinline__ void store_chunk(typename Elem<BF16>::T *row, const ChunkAt &at, int D,
                                            const float (&v)[8])
{
    if (!at.live)
        return;
    if constexpr (TINY) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < D)
                Elem<BF16>::store(row + i, v[i]);
    } else {
        store8<BF16>(row + at.off, v);
    }
}

// Sum of f(i) over the chunk's own elements.
template <bool TINY, typename F>
__device__ __forceinline__ float own_sum(const ChunkAt &at, int D, bool ragged, F f)
{
    float s = 0.f;
    if (TINY || ragged) {
        const int end = TINY ? D : kChunk;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s += (i >= at.lo && i < end) ? f(i) : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s += f(i);
    }
    return at.live ? s : 0.f;
}

}  // namespace
}  // namespace mamba
