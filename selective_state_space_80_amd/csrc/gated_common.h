// The step of the gated linear recurrence and the scan of its steps over a wave,
// shared by its forward and backward kernels.
//
//   v = c softplus(lam) sigmoid(r),  a = e^-v,  m = sqrt(1 - a^2)
//   h <- a h + m sigmoid(i) x
//
// Two things are kept from losing their digits where a is next to 1 (long memories).
// 1 - a^2 comes from a polynomial in the exponent there, not from a.  And spans of steps
// are joined with the sum of their exponents, not the product of their a: a's rounding
// there (6e-8) would add up over the steps of a sequence, as it is it adds up over a
// lane's eight.
#pragma once

#include "device_common.h"

namespace mamba {

constexpr int kLaneSteps = 8;  // consecutive steps of a row that a lane takes

typedef uint32_t gated_u32x4 __attribute__((ext_vector_type(4)));
typedef float gated_f32x4 __attribute__((ext_vector_type(4)));

// Eight consecutive elements of a row as they lie in memory.
template <bool BF16> struct Eight;
template <> struct Eight<true> {
    gated_u32x4 v;
    __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(&v, p, 16); }
    __device__ __forceinline__ float get(int j) const
    {
        return j & 1 ? __uint_as_float(v[j >> 1] & 0xffff0000u) : __uint_as_float(v[j >> 1] << 16);
    }
    __device__ __forceinline__ void fill(float f)
    {
        const uint32_t b = __float_as_uint(f) >> 16;  // 0 and -inf only: exact
        v = gated_u32x4{b | b << 16, b | b << 16, b | b << 16, b | b << 16};
    }
    __device__ __forceinline__ uint16_t raw(int j) const { return (uint16_t)(v[j >> 1] >> (16 * (j & 1))); }
    __device__ __forceinline__ void set_raw(int j, uint16_t bits)
    {
        const uint32_t w = v[j >> 1];
        v[j >> 1] = j & 1 ? (w & 0xffffu) | (uint32_t)bits << 16 : (w & 0xffff0000u) | bits;
    }
    // Rounds eight values and stores the first n of them: past the caches, which a
    // wave's whole piece of 1024 bytes gains from (8 x 5120 x 2048 forward 130 -> 125 us,
    // backward 232 -> 221; fp32's two stores of half lines lose, 1 x 1536 x 131072
    // backward 1084 -> 1251).
    static __device__ __forceinline__ void store(uint16_t *p, const float (&f)[kLaneSteps], bool whole, int n)
    {
        const gated_u32x4 w = {cvt2(f[0], f[1]), cvt2(f[2], f[3]), cvt2(f[4], f[5]), cvt2(f[6], f[7])};
        if (whole || n >= kLaneSteps) {
            typedef gated_u32x4 __attribute__((aligned(2))) loose;
            __builtin_nontemporal_store(w, (loose *)p);
        } else {
#pragma unroll
            for (int j = 0; j < kLaneSteps - 1; ++j)
                if (j < n)
                    p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
};
template <> struct Eight<false> {
    gated_f32x4 v[2];
    __device__ __forceinline__ void load(const float *p) { __builtin_memcpy(v, p, 32); }
    __device__ __forceinline__ float get(int j) const { return v[j >> 2][j & 3]; }
    __device__ __forceinline__ void fill(float f)
    {
        v[0] = gated_f32x4{f, f, f, f};
        v[1] = v[0];
    }
    __device__ __forceinline__ float raw(int j) const { return get(j); }
    __device__ __forceinline__ void set_raw(int j, float f) { v[j >> 2][j & 3] = f; }
    static __device__ __forceinline__ void store(float *p, const float (&f)[kLaneSteps], bool whole, int n)
    {
        if (whole || n >= kLaneSteps) {
            __builtin_memcpy(p, f, 32);
        } else {
#pragma unroll
            for (int j = 0; j < kLaneSteps - 1; ++j)
                if (j < n)
                    p[j] = f[j];
        }
    }
};

// Steps of a group's 8 G from `from` on that lie before L.
template <int G> __device__ __forceinline__ int steps_left(int64_t L, int64_t from)
{
    const int64_t left = L - from;
    return left <= 0 ? 0 : (left < G * kLaneSteps ? (int)left : G * kLaneSteps);
}
// A lane's share of them: its eight start at `off`.
__device__ __forceinline__ int lane_share(int left, uint32_t off)
{
    const int n = left - (int)off;
    return n <= 0 ? 0 : (n < kLaneSteps ? n : kLaneSteps);
}
// The same for every lane of a wave, which then takes what hangs on it by scalar means.
template <bool WHOLE_WAVE> __device__ __forceinline__ int uniform(int v)
{
    return WHOLE_WAVE ? __builtin_amdgcn_readfirstlane(v) : v;
}

// The first n (at most 8) elements from p on; the others are `rest`.  whole: every lane
// of the wave has all eight.  At a row's end
// the elements are loaded one by one, but all at once: those past the end repeat the
// last (with a branch for each, a row's end cost as many round trips to memory:
// 8 x 5120 x 300 bf16 56 us).
template <bool BF16>
__device__ __forceinline__ void load_some(Eight<BF16> &to, const typename Elem<BF16>::T *p, bool whole, int n, float rest)
{
    if (whole || n >= kLaneSteps) {
        to.load(p);
        return;
    }
    to.fill(rest);
    if (n > 0) {
        typename Elem<BF16>::T some[kLaneSteps - 1];
#pragma unroll
        for (int j = 0; j < kLaneSteps - 1; ++j)
            some[j] = p[j < n ? j : n - 1];
#pragma unroll
        for (int j = 0; j < kLaneSteps - 1; ++j)
            to.set_raw(j, j < n ? some[j] : to.raw(j));
    }
}

// Bit j: step j of the lane's starts a sequence.
__device__ __forceinline__ uint32_t load_resets(const uint8_t *p, bool whole, int n)
{
    uint32_t bits = 0;
    if (whole || n >= kLaneSteps) {
        uint32_t w[2];
        __builtin_memcpy(w, p, 8);
#pragma unroll
        for (int j = 0; j < kLaneSteps; ++j)
            bits |= ((w[j >> 2] >> (8 * (j & 3))) & 0xffu) != 0 ? 1u << j : 0u;
    } else {
        if (n > 0) {
            uint8_t some[kLaneSteps - 1];
#pragma unroll
            for (int j = 0; j < kLaneSteps - 1; ++j)
                some[j] = p[j < n ? j : n - 1];
#pragma unroll
            for (int j = 0; j < kLaneSteps - 1; ++j)
                bits |= j < n && some[j] != 0 ? 1u << j : 0u;
        }
    }
    return bits;
}

// 1 / (1 + 2^-(x log2 e + bias)), bias in the same units; 0 at -infinity, 1 at infinity.
__device__ __forceinline__ float sigmoid_log2(float x, float bias2)
{
    return hw_rcp(1.f + hw_exp2(fmaf(x, -kLog2e, -bias2)));
}

// ln(1 + e^x), which scales every v of a row: max(x, 0) + ln(1 + t), t = e^-|x|.  t by
// 2^x of the fraction of |x| log2 e, which the split constant gives to within 2^-25; the
// logarithm as 2 atanh(q), q = t / (2 + t) at most 1/3, whose series to q^15 is left off
// below 1e-8 relative.  |x| is held at 200, where t is 0 in fp32: of a larger one the
// product with log2 e is off by more than a fraction's range (of an infinite one there is
// none).  By a comparison, which lets a NaN through.
__device__ __forceinline__ float softplus_row(float x)
{
    constexpr float kLog2eLow = (float)(1.44269504088896340736 - (double)kLog2e);
    const float y = fabsf(x) > 200.f ? -200.f : -fabsf(x), whole = __builtin_rintf(y * kLog2e);
    const float part = fmaf(y, kLog2eLow, fmaf(y, kLog2e, -whole));
    const float t = __builtin_amdgcn_ldexpf(hw_exp2(part), (int)fmaxf(whole, -1000.f));
    const float q = t * hw_rcp(2.f + t), q2 = q * q;
    float s = 1.f / 15.f;
    s = fmaf(s, q2, 1.f / 13.f);
    s = fmaf(s, q2, 1.f / 11.f);
    s = fmaf(s, q2, 1.f / 9.f);
    s = fmaf(s, q2, 1.f / 7.f);
    s = fmaf(s, q2, 1.f / 5.f);
    s = fmaf(s, q2, 1.f / 3.f);
    s = fmaf(s, q2, 1.f);
    return fmaxf(x, 0.f) + 2.f * q * s;
}

// A row's v = rate * sigmoid(r + r_bias) and the bias of a gate, in exponents of 2.  An infinite
// one counts as the largest float, so that r = -infinity, which the steps past a row's end
// have too, makes v 0 whatever they are (0 * infinity and infinity - infinity are NaN).  By
// a comparison, which lets a NaN through.
__device__ __forceinline__ float held(float v)
{
    constexpr float kMost = 3.402823466e38f;
    return fabsf(v) > kMost ? copysignf(kMost, v) : v;
}
__device__ __forceinline__ float row_rate(float c, float lam) { return held(c * softplus_row(lam) * kLog2e); }
__device__ __forceinline__ float row_bias(float bias) { return held(bias * kLog2e); }

// 1 - a^2 for a = 2^-u, u >= 0.  Below 1/8 by a polynomial in u (through (1 - 2^-2u) / u at
// the interval's Chebyshev points; off by 1e-8 relative at most); above, the subtraction
// keeps all but three bits.
__device__ __forceinline__ float square_of(float u, float a)
{
    float p = 0.0397070758f;
    p = fmaf(p, u, -0.153570428f);
    p = fmaf(p, u, 0.444018692f);
    p = fmaf(p, u, -0.96090579f);
    p = fmaf(p, u, 1.38629436f);
    return u < 0.125f ? u * p : fmaf(-a, a, 1.f);
}

// The value of the lane that the DPP control names, 0 where there is none or the row
// of 16 is not in ROWS.
template <int CTRL, int ROWS = 0xf> __device__ __forceinline__ float lane_of(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}
constexpr int kRowShr = 0x110, kRowShl = 0x100, kWaveShr1 = 0x138, kWaveShl1 = 0x130, kBcast15 = 0x142,
              kBcast31 = 0x143;

__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// A span's map s -> 2^-U s + S.  `after`: this one behind another.  With DROPS a map
// of U = infinity (a reset) drops even a NaN or an infinity of what lies before it.  The
// exponents of a lane's steps are held at 1e30, so that no sum of them comes to that.
template <bool DROPS> struct Span {
    float U, S;
    __device__ __forceinline__ float of(float s) const
    {
        const float v = fmaf(hw_exp2(-U), s, S);
        return DROPS && U == __builtin_inff() ? S : v;
    }
    __device__ __forceinline__ void after(const Span &before)
    {
        S = of(before.S);
        U = DROPS && U == __builtin_inff() ? U : U + before.U;
    }
};

template <bool DROPS> __device__ __forceinline__ Span<DROPS> lane_span(float U, bool reset, float S)
{
    if constexpr (DROPS)
        U = reset ? __builtin_inff() : fminf(U, 1e30f);  // of a NaN too: S is one then
    return {U, S};
}

template <int CTRL, int ROWS = 0xf, bool DROPS>
__device__ __forceinline__ Span<DROPS> span_of_lane(const Span<DROPS> &m)
{
    return {lane_of<CTRL, ROWS>(m.U), lane_of<CTRL, ROWS>(m.S)};
}
template <bool DROPS> __device__ __forceinline__ Span<DROPS> read_span(const Span<DROPS> &m, int lane)
{
    return {read_lane(m.U, lane), read_lane(m.S, lane)};
}

// Joins to each lane's span those of the lanes before it (of its group of G lanes);
// returns the join without the lane's own.
template <int G, bool DROPS> __device__ __forceinline__ Span<DROPS> join_before(Span<DROPS> &m)
{
    const Span<DROPS> none{0.f, 0.f};
    const int in = threadIdx.x & (G - 1);
    if constexpr (G >= 16) {
        m.after(span_of_lane<kRowShr + 1>(m));
        m.after(span_of_lane<kRowShr + 2>(m));
        m.after(span_of_lane<kRowShr + 4>(m));
        m.after(span_of_lane<kRowShr + 8>(m));
        if constexpr (G >= 32)
            m.after(span_of_lane<kBcast15, 0xa>(m));
        if constexpr (G == 64)
            m.after(span_of_lane<kBcast31, 0xc>(m));
    } else {
        static_assert(G == 4, "groups of 4, 16, 32 or 64 lanes");
        const Span<DROPS> p = span_of_lane<kRowShr + 1>(m);
        m.after(in >= 1 ? p : none);
        const Span<DROPS> q = span_of_lane<kRowShr + 2>(m);
        m.after(in >= 2 ? q : none);
    }
    const Span<DROPS> e = span_of_lane<kWaveShr1>(m);
    return G == 64 || in > 0 ? e : none;
}

// The same from the other end: the spans of the lanes behind each lane.
template <int G, bool DROPS> __device__ __forceinline__ Span<DROPS> join_behind(Span<DROPS> &m)
{
    const Span<DROPS> none{0.f, 0.f};
    const int lane = threadIdx.x & 63, in = lane & (G - 1);
    if constexpr (G >= 16) {
        m.after(span_of_lane<kRowShl + 1>(m));
        m.after(span_of_lane<kRowShl + 2>(m));
        m.after(span_of_lane<kRowShl + 4>(m));
        m.after(span_of_lane<kRowShl + 8>(m));
        if constexpr (G >= 32) {  // rows of 16: their spans are in their first lanes
            const Span<DROPS> r1 = read_span(m, 16), r3 = read_span(m, 48);
            const int row = lane >> 4;
            if constexpr (G == 64) {
                Span<DROPS> r23 = read_span(m, 32);
                r23.after(r3);
                Span<DROPS> r123 = r1;
                r123.after(r23);
                m.after(row == 0 ? r123 : (row == 1 ? r23 : (row == 2 ? r3 : none)));
            } else {
                m.after(row == 0 ? r1 : (row == 2 ? r3 : none));
            }
        }
    } else {
        static_assert(G == 4, "groups of 4, 16, 32 or 64 lanes");
        const Span<DROPS> p = span_of_lane<kRowShl + 1>(m);
        m.after(in <= 2 ? p : none);
        const Span<DROPS> q = span_of_lane<kRowShl + 2>(m);
        m.after(in <= 1 ? q : none);
    }
    const Span<DROPS> e = span_of_lane<kWaveShl1>(m);
    return G == 64 || in < G - 1 ? e : none;
}

// The map of a row's parts before this one (lane l holds part l's, or nothing), joined,
// applied to the state that enters the first.
template <bool DROPS>
__device__ __forceinline__ float through_parts(const float2 *maps, int count, bool from_end, int parts, float s)
{
    const int lane = threadIdx.x & 63;
    Span<DROPS> m{0.f, 0.f};
    if (lane < count) {
        const float2 f = maps[from_end ? parts - 1 - lane : lane];
        m = Span<DROPS>{f.x, f.y};
    }
    join_before<64, DROPS>(m);
    return read_span(m, 63).of(s);
}

// Threads of a workgroup: one row where several waves share it, which meet in LDS.
constexpr int gated_threads(int waves) { return waves == 1 ? 256 : 64 * waves; }

// Lanes a row of L steps takes.
inline int gated_group(int64_t L)
{
    return L <= 4 * kLaneSteps ? 4 : (L <= 16 * kLaneSteps ? 16 : (L <= 32 * kLaneSteps ? 32 : 64));
}

// Waves that share a row: at most `most`, while there are fewer than about 12000 waves
// in all and each has four chunks of the row or more (a power of two).
inline int gated_waves(int64_t rows, int64_t L, int most)
{
    const int64_t chunks = (L + 64 * kLaneSteps - 1) / (64 * kLaneSteps);
    int waves = 1;
    while (waves * 2 <= most && waves * 2 * rows <= 12288 && waves * 2 * 4 <= chunks)
        waves *= 2;
    return waves;
}

}  // namespace mamba
