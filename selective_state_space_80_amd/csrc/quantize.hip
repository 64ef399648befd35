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
// Fewer tiles, or more channels than the registers of 64-byte tiles hold, take
// tiles of 32 or 16 bytes (PARTS); sequences shorter than 16 bytes have a kernel
// of their own.
//
// Bound by memory.  8 x 5120 x 2048 bf16 (252 MB) takes 44 us (5.7 TB/s) with
// the input in the last-level cache, where a scan has just left it, and 69 us
// from memory: there is room for one workgroup a CU, so its loads do not
// overlap its stores.  1 x 1536 x 131072 bf16 (604 MB) takes 135 us;
// 64 x 5120 x 4 bf16 3.6 us, bound by its launch and its two dependent waits.
// (Times in this file are from memory, inputs taken in turn, unless said.)
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

// Of fewer than four channels (SHORT), tokens are read one by one, the index
// held below the `left` there are; otherwise the last 16 bytes are moved back
// to end with the sequence.
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

// Which tile a workgroup takes.  Neighbouring tiles read parts of the same cache
// lines, so each of the 8 XCDs (workgroups go to them in turn) takes a
// contiguous share.  What is in flight should also touch every memory channel
// alike.  They alternate within 4 KB, and a tile reads the same few bytes of
// each: so each XCD starts an eighth of its share after the one before, and
// where rows repeat every 4 KB, the 64-byte tiles (about 32 of an XCD run at
// once) go first by every second pair and then by the others.  8 x 5120 x 2048
// bf16 74 us without either, 74 with the first, 69 with both; fp32 112, 100,
// 103; 2 x 5120 x 4096 fp32 64, 60, 54; 8 x 8192 x 2048 bf16, in 32-byte tiles,
// 147 and 128.
template <int PARTS> __device__ __forceinline__ int64_t tile_of(int64_t row_bytes)
{
    const int64_t all = gridDim.x, xcd = blockIdx.x % 8, more = all % 8;
    const int64_t share = all / 8 + (xcd < more ? 1 : 0);
    int64_t i = blockIdx.x / 8;
    if (PARTS == 4 && row_bytes % 4096 == 0 && (i | 63) < share) {
        const int64_t pair = i % 32 / 2, half = i % 64 / 32;
        i = i / 64 * 64 + pair * 4 + half * 2 + i % 2;
    }
    i += share / 8 * xcd;
    if (i >= share)
        i -= share;
    return xcd * (all / 8) + (xcd < more ? xcd : more) + i;
}

// HELD groups of channels stay in registers; 0: they are more than that, and
// the second pass reads them again.
template <bool BF16, int PARTS, int THREADS, int HELD, bool SHORT>
__global__ __launch_bounds__(THREADS) void quantize_channel_kernel(const ChannelParams p)
{
    using T = typename Elem<BF16>::T;
    using Tok = Tokens<BF16>;
    constexpr int kTok = Tok::kCount, kTile = PARTS * kTok;
    __shared__ uint32_t tops[THREADS / 64][PARTS][4];
    __shared__ RowScale<BF16> rows[kTile];
    __shared__ int special;  // a row is raised, or not finite
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n_waves = blockDim.x >> 6;
    const int64_t group = blockDim.x / PARTS * kChan;  // channels
    const int part = lane & (PARTS - 1);          // which 16 bytes of the tokens
    const int64_t c0 = (int64_t)(threadIdx.x / PARTS) * kChan;  // first of its channels
    const int64_t tile = tile_of<PARTS>(p.L * (int64_t)sizeof(T));
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
    // over the lanes of the same tokens (lane % PARTS), then over the waves
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (PARTS == 1)
            top[i] = max_abs<BF16>(top[i], dpp<0x121>(top[i]));  // row rotated by 1
        if constexpr (PARTS <= 2)
            top[i] = max_abs<BF16>(top[i], dpp<0x122>(top[i]));  // by 2
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
        const RowScale<BF16> rs(t);
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
    // Where the registers are full, a token's fp64 multiplier is read when it is
    // needed (8 x 6144 x 2048 fp32: 125 us; held, other values spill, 131).
    constexpr bool kReread = !BF16 && HELD == kMaxHeld;
    RowScale<BF16> row[kTok];
    if constexpr (!kReread) {
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            row[i].mul = rows[part * kTok + i].mul;
    }
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
            if constexpr (kReread) {
                int at = part * kTok + i;
                asm volatile("" : "+v"(at));
                row[i].mul = rows[at].mul;
            }
            uint32_t byte[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = t[r].get(i);
                if (any_special)
                    v *= rows[part * kTok + i].raise;
                byte[r] = row[i].nearest(v);
            }
            uint32_t w = pack4(byte);
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

// Sequences of L tokens that are shorter than 16 bytes: a workgroup takes one,
// and a thread all tokens of four neighbouring channels, which lie one after
// another.  Two groups of channels stay in registers; where there are more
// (MANY), the second pass reads them again.
template <bool BF16, int L, bool MANY>
__global__ __launch_bounds__(kMostThreads) void quantize_short_kernel(const ChannelParams p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kHeld = 2, kWords = (BF16 ? 2 : 4) * L;
    struct Piece {
        uint32_t v[kWords];
        __device__ __forceinline__ float get(int e) const
        {
            if constexpr (BF16)
                return __uint_as_float(e % 2 ? v[e / 2] & 0xffff0000u : v[e / 2] << 16);
            else
                return __uint_as_float(v[e]);
        }
    };
    __shared__ uint32_t tops[kMostThreads / 64][L];
    __shared__ RowScale<BF16> rows[L];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n_waves = blockDim.x >> 6;
    const int64_t b = blockIdx.x;
    const int64_t group = (int64_t)blockDim.x * kChan;
    const T *x = (const T *)p.x + b * p.K * L;
    // the last four channels are moved back to end with K
    auto channel = [&](int64_t g) {
        const int64_t c = g * group + (int64_t)threadIdx.x * kChan;
        return c + kChan <= p.K ? c : p.K - kChan;
    };
    auto load = [&](Piece &t, int64_t g) { __builtin_memcpy(t.v, x + channel(g) * L, kWords * 4); };
    const int64_t groups = (p.K + group - 1) / group;

    uint32_t top[L];
#pragma unroll
    for (int i = 0; i < L; ++i)
        top[i] = 0;
    auto take = [&](const Piece &t) {
#pragma unroll
        for (int e = 0; e < kChan * L; ++e)
            top[e % L] = umax(top[e % L], abs_bits(t.get(e)));
    };
    Piece held[kHeld];
#pragma unroll
    for (int g = 0; g < kHeld; ++g)
        load(held[g], g);
#pragma unroll
    for (int g = 0; g < kHeld; ++g)
        take(held[g]);
    if constexpr (MANY) {
#pragma unroll 2
        for (int64_t g = kHeld; g < groups; ++g) {
            Piece t;
            load(t, g);
            take(t);
        }
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const uint32_t t = lane_max<64>(top[i]);
        if (lane == 0)
            tops[wave][i] = t;
    }
    __syncthreads();
    if (threadIdx.x < L) {
        uint32_t t = 0;
        for (int w = 0; w < n_waves; ++w)
            t = umax(t, tops[w][threadIdx.x]);
        const RowScale<BF16> rs(t);
        rows[threadIdx.x] = rs;
        p.scale[b * L + threadIdx.x] = rs.scale;
    }
    __syncthreads();
    int8_t *q = p.q + b * L * p.K;
    auto put = [&](const Piece &t, int64_t g) {
        const int64_t c = channel(g);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            uint32_t byte[kChan];
#pragma unroll
            for (int r = 0; r < kChan; ++r)
                byte[r] = rows[i].nearest(t.get(r * L + i) * rows[i].raise);
            const uint32_t w = pack4(byte) & rows[i].mask;
            __builtin_memcpy(q + i * p.K + c, &w, 4);
        }
    };
#pragma unroll
    for (int g = 0; g < kHeld; ++g)
        put(held[g], g);
    if constexpr (MANY) {
        for (int64_t g = kHeld; g < groups; ++g) {
            Piece t;
            load(t, g);
            put(t, g);
        }
    }
}

template <bool BF16, int L> hipError_t start_short(const QuantChannelArgs &a, hipStream_t s)
{
    if constexpr (L < Tokens<BF16>::kCount - 1) {
        if (a.L != L)
            return start_short<BF16, L + 1>(a, s);
    }
    const ChannelParams p{a.x, a.q, a.scale, a.L, a.K, 1};
    const int64_t quads = (a.K + kChan - 1) / kChan;
    const bool many = quads > 2 * kMostThreads;
    const int64_t threads = many ? kMostThreads : ((quads + 1) / 2 + 63) / 64 * 64;
    const dim3 grid((unsigned)a.B), block((unsigned)threads);
    if (many)
        quantize_short_kernel<BF16, L, true><<<grid, block, 0, s>>>(p);
    else if constexpr (L > 1)  // single tokens of fewer channels are rows of the token-major form
        quantize_short_kernel<BF16, L, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

// The form that holds `groups` groups, of those that calls reach.
template <bool BF16, int PARTS, int THREADS, int HELD>
void start_held(int64_t groups, dim3 grid, dim3 block, const ChannelParams &p, hipStream_t s)
{
    constexpr int kFewest = THREADS / PARTS * kChan == kMostThreads ? 1 : kMaxHeld / 2 + 1;
    if constexpr (HELD > kFewest) {
        if (groups < HELD)
            return start_held<BF16, PARTS, THREADS, HELD - 1>(groups, grid, block, p, s);
    }
    quantize_channel_kernel<BF16, PARTS, THREADS, HELD, false><<<grid, block, 0, s>>>(p);
}

template <bool BF16, int PARTS, int THREADS> hipError_t start(const QuantChannelArgs &a, hipStream_t s)
{
    constexpr int kTok = Tokens<BF16>::kCount, kMostGroup = THREADS / PARTS * kChan;
    const int64_t tiles = (a.L + PARTS * kTok - 1) / (PARTS * kTok);
    const ChannelParams p{a.x, a.q, a.scale, a.L, a.K, tiles};
    // as few groups as there can be, then as few waves as those need
    const int64_t groups = (a.K + kMostGroup - 1) / kMostGroup;
    const int64_t threads = (a.K + groups * kChan - 1) / (groups * kChan) * PARTS;
    const dim3 grid((unsigned)(a.B * tiles)), block((unsigned)((threads + 63) / 64 * 64));
    if (groups <= kMaxHeld) {
        start_held<BF16, PARTS, THREADS, kMaxHeld>(groups, grid, block, p, s);
    } else if constexpr (PARTS == 4) {
        quantize_channel_kernel<BF16, PARTS, THREADS, 0, false><<<grid, block, 0, s>>>(p);
    }
    return hipGetLastError();
}

template <bool BF16> hipError_t dispatch(const QuantChannelArgs &a, hipStream_t s)
{
    constexpr int kTok = Tokens<BF16>::kCount;
    constexpr int64_t kHeldChannels = kMaxHeld * kMostThreads;
    const int64_t tiles = a.B * ((a.L + 4 * kTok - 1) / (4 * kTok));
    if (a.K < kChan) {
        const ChannelParams p{a.x, a.q, a.scale, a.L, a.K, (a.L + 4 * kTok - 1) / (4 * kTok)};
        quantize_channel_kernel<BF16, 4, kMostThreads, 0, true><<<dim3((unsigned)tiles), dim3(64), 0, s>>>(p);
        return hipGetLastError();
    }
    // Whole tiles take over from 16 bytes on (64 x 5120 x 7 bf16 5.1 us so and
    // 64 x 5120 x 8 6.8; x 7 token by token 31.6).
    if (a.L < kTok)
        return start_short<BF16, 1>(a, s);
    // Few tiles leave most CUs idle: below half a tile a CU, tiles of 16 bytes by a
    // quarter of the threads (bf16, in us, so and in tiles of 64 bytes: 1 x 5120 x
    // 1000 11.4 and 16.9; 2 x 5120 x 1024 13.1 and 18.8; 1 x 5120 x 3000 23.4 and
    // 25.4; but 4000 24.7 and 23.4; 8000 44 and 30).
    if (a.K <= kHeldChannels)
        return tiles < 128 ? start<BF16, 1, kMostThreads / 4>(a, s) : start<BF16, 4, kMostThreads>(a, s);
    // More channels are held by smaller tiles of as many threads, up to the most
    // that registers hold; read twice instead, 1 x 20000 x 1000 bf16 takes 109 us
    // (41 so), 8 x 8192 x 2048 144 (128; fp32 239 and 189), 2 x 16384 x 2048 120
    // (76; fp32 148 and 133).
    if (a.K <= 2 * kHeldChannels)
        return start<BF16, 2, kMostThreads>(a, s);
    if (a.K <= 4 * kHeldChannels)
        return start<BF16, 1, kMostThreads>(a, s);
    return start<BF16, 4, kMostThreads>(a, s);
}

}  // namespace

hipError_t launch_quantize_channel_major(const QuantChannelArgs &a, hipStream_t s)
{
    return a.bf16 ? dispatch<true>(a, s) : dispatch<false>(a, s);
}

}  // namespace mamba
