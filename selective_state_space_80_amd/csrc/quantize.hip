// 8-bit quantisation of channel-major activations, as the scans write them:
// x [B, K, L] -> q [B, L, K] with one scale per token (b, l), the row scale of
// the token-major form:  scale = max_k|x| / 127,  q = rne(x * 127 / max_k|x|).
//
// A workgroup takes 64 tokens of one sequence: a first pass over the K channels
// finds each token's largest value, a second reads the same tile again (from
// the caches, where it still lies) and writes it transposed through LDS.
#include <hip/hip_runtime.h>

#include "quant.h"
#include "row_chunk.h"

namespace mamba {
namespace {

constexpr int kTok = 64;        // tokens of a workgroup
constexpr int kChan = 128;      // channels transposed at a time
constexpr int kThreads = 512;

struct ChannelParams {
    const void *x;
    int8_t *q;
    float *scale;
    int64_t L, K, tiles;
};

template <bool BF16> __global__ __launch_bounds__(kThreads) void quantize_channel_kernel(const ChannelParams p)
{
    using T = typename Elem<BF16>::T;
    __shared__ uint32_t top[kTok];
    __shared__ int8_t tile[kTok][kChan + 4];
    const int tok = threadIdx.x & 63, sub = threadIdx.x >> 6;
    const int64_t b = blockIdx.x / p.tiles, l0 = (int64_t)(blockIdx.x % p.tiles) * kTok;
    const int64_t l = l0 + tok < p.L ? l0 + tok : p.L - 1;
    const T *col = (const T *)p.x + b * p.K * p.L + l;
    if (threadIdx.x < kTok)
        top[threadIdx.x] = 0;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll 8
    for (int64_t k = sub; k < p.K; k += kThreads / 64)
        m = umax(m, abs_bits(Elem<BF16>::load(col + k * p.L)));
    atomicMax(&top[tok], m);  // a maximum: the order does not matter
    __syncthreads();
    const RowScale rs = row_scale(top[tok]);
    if (sub == 0 && l0 + tok < p.L)
        p.scale[b * p.L + l0 + tok] = rs.scale;
    for (int64_t k0 = 0; k0 < p.K; k0 += kChan) {
#pragma unroll
        for (int c = sub; c < kChan; c += kThreads / 64) {
            const int64_t k = k0 + c < p.K ? k0 + c : p.K - 1;
            const float v = Elem<BF16>::load(col + k * p.L) * rs.raise;
            tile[tok][c] = (int8_t)(__float_as_uint(fmaf(v, rs.mul, 12582912.f)) & rs.mask);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kTok * kChan; i += kThreads) {
            const int t = i / kChan, c = i % kChan;
            if (l0 + t < p.L && k0 + c < p.K)
                p.q[(b * p.L + l0 + t) * p.K + k0 + c] = tile[t][c];
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_quantize_channel_major(const QuantChannelArgs &a, hipStream_t s)
{
    const int64_t tiles = (a.L + kTok - 1) / kTok;
    ChannelParams p{a.x, a.q, a.scale, a.L, a.K, tiles};
    const dim3 grid((unsigned)(a.B * tiles));
    if (a.bf16)
        quantize_channel_kernel<true><<<grid, dim3(kThreads), 0, s>>>(p);
    else
        quantize_channel_kernel<false><<<grid, dim3(kThreads), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace mamba
