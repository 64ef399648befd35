// 8-bit quantisation of channel-major activations, as the scans write them:
// x [B, K, L] -> q [B, L, K] with one scale per token (b, l), the row scale of
// the token-major form:  scale = max_k|x| / 127,  q = rne(x * 127 / max_k|x|).
//
// A scale needs all K channels of its token before the first of them can be
// written.  A workgroup takes 64 bytes of tokens (32 bf16 or 16 fp32) of one
// sequence and holds all their channels in registers, packed as loaded, so the
// input is read once: 320 KB of the CU's 512 KB at K = 5120.  A thread has 16
// bytes of tokens of four neighbouring channels per group of as many channels
// as the workgroup has threads (up to 1024: one wave for 64 channels, five
// groups of 1024 for 5120); the four bytes it makes of a token are one 4-byte
// store, and 16 lanes' stores are 64 neighbouring bytes: the transposition
// needs no LDS.
//
// Bound by memory.  8 x 5120 x 2048 bf16 (252 MB) takes 45 us (5.5 TB/s) with
// the input in the last-level cache, where a scan has just left it, and 73 us
// from memory: there is room for one workgroup a CU, so its loads do not
// overlap its stores (64 without the stores, 70 and 99 us before neighbouring
// tiles shared an XCD's L2).  1 x 1536 x 131072 bf16 (604 MB) takes 143 us.
#include <hip/hip_runtime.h>

#include "quant.h"
#include "row_chunk.h"

namespace mamba {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kChan = 4;     // neighbouring channels of a thread
constexpr int kMaxHeld = 6;  // groups held in registers (96 of the 128 there are)

struct ChannelParams {
    const void *x;
    int8_t *q;
    float *scale;
    int64_t L, K, tiles;
};

// 16 bytes of a channel's tokens, as loaded.
template <bool BF16> struct Tokens {
    static constexpr int kCount = BF16 ? 8 : 4;
    u32x4 v;
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (BF16)
            return __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
        else
            return __uint_as_float(v[i]);
    }
};

// Sequences shorter than 16 bytes, and fewer than four channels (SHORT), are
// read token by token, the index held below the `left` there are; otherwise the
// last 16 bytes are moved back to end with the sequence.
template <bool BF16, bool SHORT>
__device__ __forceinline__ Tokens<BF16> load_tokens(const typename Elem<BF16>::T *channel, int left)
{
    Tokens<BF16> t;
    if constexpr (SHORT) {
        t.v = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Tokens<BF16>::kCount; ++i) {
            const uint32_t e = BF16 ? (uint32_t)((const uint16_t *)channel)[i < left ? i : left - 1]
                                    : ((const uint32_t *)channel)[i < left ? i : left - 1];
            t.v[BF16 ? i / 2 : i] |= BF16 && i % 2 ? e << 16 : e;
        }
    } else {
        __builtin_memcpy(&t.v, channel, 16);
    }
    return t;
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Larger of the |values| of two words: two bf16 halves, or one fp32 (the bits
// of |v| order as |v|, NaN above all).
template <bool BF16> __device__ __forceinline__ uint32_t max_abs(uint32_t top, uint32_t v)
{
    if constexpr (BF16) {
        const u16x2 a = __builtin_bit_cast(u16x2, top), b = __builtin_bit_cast(u16x2, v & 0x7fff7fffu);
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
    } else {
        return umax(top, v & 0x7fffffffu);
    }
}

// HELD groups of channels stay in registers; 0: they are more than that, and
// the second pass reads them again.
template <bool BF16, int PARTS, int HELD, bool SHORT>
__global__ __launch_bounds__(kMostThreads / 4 * PARTS) void quantize_channel_kernel(const ChannelParams p)
{
    using T = typename Elem<BF16>::T;
    using Tok = Tokens<BF16>;
    constexpr int kTok = Tok::kCount, kTile = PARTS * kTok;
    __shared__ uint32_t tops[kMostThreads / 256 * PARTS][PARTS][4];
    __shared__ RowScale rows[kTile];
    __shared__ int special;  // a row is raised, or not finite
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n_waves = blockDim.x >> 6;
    const int64_t group = blockDim.x / PARTS * kChan;  // channels
    const int part = lane & (PARTS - 1);          // which 16 bytes of the tokens
    const int64_t c0 = (int64_t)(threadIdx.x / PARTS) * kChan;  // first of its channels
    // Neighbouring tiles read the two halves of the same cache lines: each of
    // the 8 XCDs (workgroups go to them in turn) takes a contiguous share.
    const int64_t all = gridDim.x, xcd = blockIdx.x % 8, more = all % 8;
    const int64_t tile = xcd * (all / 8) + (xcd < more ? xcd : more) + blockIdx.x / 8;
    const int64_t b = tile / p.tiles, l0 = (tile % p.tiles) * kTile;
    const int64_t to = l0 + part * kTok;
    const int64_t l = SHORT ? (to < p.L ? to : p.L - 1) : (to + kTok <= p.L ? to : p.L - kTok);
    const bool live = to < p.L;
    const int left = SHORT ? (int)(p.L - l < kTok ? p.L - l : kTok) : kTok;  // tokens there are
    const T *x = (const T *)p.x + b * p.K * p.L + l;
    // The four channels of a thread and group; the last ones are moved back to
    // end with K (threads then make the same bytes twice).  Below four channels
    // (SHORT) they repeat the last.
    auto channel = [&](int64_t g) {
        const int64_t c = g * group + c0;
        return SHORT || c + kChan <= p.K ? c : p.K - kChan;
    };
    auto load4 = [&](Tok(&t)[kChan], int64_t g) {
        const int64_t c = channel(g);
        if constexpr (SHORT) {
#pragma unroll
            for (int r = 0; r < kChan; ++r)
                t[r] = load_tokens<BF16, true>(x + (c + r < p.K ? c + r : p.K - 1) * p.L, left);
        } else {
            const T *from = x + c * p.L;
#pragma unroll
            for (int r = 0; r < kChan; ++r, from += p.L)
                t[r] = load_tokens<BF16, false>(from, left);
        }
    };
    const int64_t groups = (p.K + group - 1) / group;

    if (threadIdx.x == 0)
        special = 0;
    Tok held[HELD ? HELD : 1][kChan];
    u32x4 top = {0, 0, 0, 0};
    if constexpr (HELD > 0) {
#pragma unroll
        for (int g = 0; g < HELD; ++g)
            load4(held[g], g);
#pragma unroll
        for (int g = 0; g < HELD; ++g)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top[i] = max_abs<BF16>(top[i], held[g][r].v[i]);
    } else {
#pragma unroll 2
        for (int64_t g = 0; g < groups; ++g) {
            Tok t[kChan];
            load4(t, g);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top[i] = max_abs<BF16>(top[i], t[r].v[i]);
        }
    }
    // over the lanes of the same tokens (lane % 4), then over the waves
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (PARTS == 2)
            top[i] = max_abs<BF16>(top[i], dpp<0x122>(top[i]));  // row rotated by 2
        top[i] = max_abs<BF16>(top[i], dpp<0x124>(top[i]));  // by 4
        top[i] = max_abs<BF16>(top[i], dpp<0x128>(top[i]));  // by 8
        top[i] = max_abs<BF16>(top[i], (uint32_t)__shfl_xor((int)top[i], 16));
        top[i] = max_abs<BF16>(top[i], (uint32_t)__shfl_xor((int)top[i], 32));
        if (lane < PARTS)
            tops[wave][part][i] = top[i];
    }
    __syncthreads();
    if (threadIdx.x < kTile) {
        const int pt = threadIdx.x / kTok, i = threadIdx.x % kTok;
        uint32_t t = 0;
        for (int w = 0; w < n_waves; ++w)
            t = max_abs<BF16>(t, tops[w][pt][BF16 ? i / 2 : i]);
        if constexpr (BF16)
            t = (i % 2 ? t >> 16 : t & 0xffffu) << 16;
        const RowScale rs = row_scale(t);
        rows[threadIdx.x] = rs;
        if (rs.raise != 1.f || rs.mask == 0)
            atomicOr(&special, 1);
        const int64_t from = l0 + pt * kTok;
        const int64_t tok = (SHORT || from + kTok <= p.L ? from : p.L - kTok) + i;
        if (from < p.L && tok < p.L)
            p.scale[b * p.L + tok] = rs.scale;
    }
    __syncthreads();
    if (!live)
        return;
    float mul[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i)
        mul[i] = rows[part * kTok + i].mul;
    const bool any_special = special != 0;
    int8_t *q = p.q + (b * p.L + l) * p.K;
    auto put = [&](const Tok(&t)[kChan], int64_t g) {
        const int64_t c = channel(g);
        if (SHORT && c >= p.K)
            return;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (SHORT && i >= left)
                continue;
            uint32_t byte[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = t[r].get(i);
                if (any_special)
                    v *= rows[part * kTok + i].raise;
                byte[r] = __float_as_uint(fmaf(v, mul[i], 12582912.f));
            }
            const uint32_t lo = __builtin_amdgcn_perm(byte[1], byte[0], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(byte[3], byte[2], 0x0c0c0400u);
            uint32_t w = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
            if (any_special)
                w &= rows[part * kTok + i].mask;
            int8_t *o = q + i * p.K + c;
            if (!SHORT || c + kChan <= p.K) {
                __builtin_memcpy(o, &w, 4);
            } else {
#pragma unroll
                for (int r = 0; r < 3; ++r)
                    if (c + r < p.K)
                        o[r] = (int8_t)(w >> (8 * r));
            }
        }
    };
    if constexpr (HELD > 0) {
#pragma unroll
        for (int g = 0; g < HELD; ++g)
            put(held[g], g);
    } else {
        for (int64_t g = 0; g < groups; ++g) {
            Tok t[kChan];
            load4(t, g);
            put(t, g);
        }
    }
}

template <bool BF16, int PARTS> hipError_t start(const QuantChannelArgs &a, hipStream_t s)
{
    constexpr int kTok = Tokens<BF16>::kCount, kMostGroup = kMostThreads;
    const int64_t tiles = (a.L + PARTS * kTok - 1) / (PARTS * kTok);
    const ChannelParams p{a.x, a.q, a.scale, a.L, a.K, tiles};
    // as few groups as there can be, then as few waves as those need
    const int64_t groups = (a.K + kMostGroup - 1) / kMostGroup;
    const int64_t threads = (a.K + groups * kChan - 1) / (groups * kChan) * PARTS;
    const dim3 grid((unsigned)(a.B * tiles)), block((unsigned)((threads + 63) / 64 * 64));
    if (a.L < kTok || a.K < kChan) {
        quantize_channel_kernel<BF16, PARTS, 0, true><<<grid, block, 0, s>>>(p);
        return hipGetLastError();
    }
    switch (groups) {
    case 1: quantize_channel_kernel<BF16, PARTS, 1, false><<<grid, block, 0, s>>>(p); break;
    case 2: quantize_channel_kernel<BF16, PARTS, 2, false><<<grid, block, 0, s>>>(p); break;
    case 3: quantize_channel_kernel<BF16, PARTS, 3, false><<<grid, block, 0, s>>>(p); break;
    case 4: quantize_channel_kernel<BF16, PARTS, 4, false><<<grid, block, 0, s>>>(p); break;
    case 5: quantize_channel_kernel<BF16, PARTS, 5, false><<<grid, block, 0, s>>>(p); break;
    case kMaxHeld: quantize_channel_kernel<BF16, PARTS, kMaxHeld, false><<<grid, block, 0, s>>>(p); break;
    default: quantize_channel_kernel<BF16, PARTS, 0, false><<<grid, block, 0, s>>>(p); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_channel_major(const QuantChannelArgs &a, hipStream_t s)
{
    // With fewer tiles than half the CUs, tiles of half the tokens by half the
    // threads: 1 x 5120 x 1000 bf16 13.9 us instead of 16.6, 64 x 5120 x 8 8.1
    // instead of 10.0; the other way 8 x 5120 x 2048 73 instead of 80.
    const int64_t per_tile = 4 * (a.bf16 ? Tokens<true>::kCount : Tokens<false>::kCount);
    if (a.B * ((a.L + per_tile - 1) / per_tile) < 128)
        return a.bf16 ? start<true, 2>(a, s) : start<false, 2>(a, s);
    return a.bf16 ? start<true, 4>(a, s) : start<false, 4>(a, s);
}

}  // namespace mamba
