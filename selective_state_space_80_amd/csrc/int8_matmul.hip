// Matrix product of 8-bit integers with a scale for each row of both operands:
//   out[m, n] = a_scale[m] b_scale[n] sum_k a[m, k] b[n, k]
// The sum is exact (32-bit integers); it is converted to fp32, scaled, and
// rounded once to the output type.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "quant.h"

namespace mamba {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 128;   // rows of each operand in a workgroup's tile
constexpr int kStep = 128;   // bytes of the inner axis a step takes

struct MatmulParams {
    const int8_t *a, *b;
    const float *a_scale, *b_scale;
    void *out;
    int64_t M, N, K;
    int64_t a_batch, b_batch;  // rows between batches: 0 = shared
    int64_t tiles_m, tiles_n;
};

// 16 bytes of a row at any address, zero past the end of the row.
__device__ __forceinline__ i32x4 load16(const int8_t *row, int64_t k, int64_t K)
{
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K) {
        uint32_t w[4] = {0, 0, 0, 0};
        for (int i = 0; i < (int)(K - k); ++i)
            w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << (8 * (i % 4));
        v = i32x4{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
    }
    return v;
}

// Place of a 16-byte chunk in a tile of 128-byte rows: the chunks of a row are
// permuted by its number, so that 16 rows read at one chunk index touch all
// 64 banks once.
__device__ __forceinline__ int slot(int row, int chunk) { return row * 8 + (chunk ^ ((row >> 1) & 7)); }

template <bool BF16> __global__ __launch_bounds__(256) void int8_matmul_kernel(const MatmulParams p)
{
    __shared__ i32x4 sa[kTile * 8], sb[kTile * 8];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    int64_t t = blockIdx.x;
    const int64_t tm = t % p.tiles_m;
    t /= p.tiles_m;
    const int64_t tn = t % p.tiles_n, batch = t / p.tiles_n;
    const int64_t m0 = tm * kTile, n0 = tn * kTile;
    const int8_t *a = p.a + batch * p.a_batch * p.K;
    const int8_t *b = p.b + batch * p.b_batch * p.K;

    i32x16 acc[2][2] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += kStep) {
        i32x4 ra[4], rb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = threadIdx.x + i * 256, row = c >> 3;
            const int64_t k = k0 + (c & 7) * 16;
            const int64_t m = m0 + row < p.M ? m0 + row : p.M - 1;
            const int64_t n = n0 + row < p.N ? n0 + row : p.N - 1;
            ra[i] = load16(a + m * p.K, k, p.K);
            rb[i] = load16(b + n * p.K, k, p.K);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = threadIdx.x + i * 256;
            sa[slot(c >> 3, c & 7)] = ra[i];
            sb[slot(c >> 3, c & 7)] = rb[i];
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            i32x4 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = sa[slot(wm + i * 32 + (lane & 31), kk * 2 + (lane >> 5))];
                fb[i] = sb[slot(wn + i * 32 + (lane & 31), kk * 2 + (lane >> 5))];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    }
    // a lane holds one m and four runs of four consecutive n per 32 x 32 block
    using T = typename Elem<BF16>::T;
    const float *asc = p.a_scale + batch * p.a_batch, *bsc = p.b_scale + batch * p.b_batch;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t m = m0 + wm + i * 32 + (lane & 31);
        if (m >= p.M)
            continue;
        const float s = asc[m];
        T *row = (T *)p.out + (batch * p.M + m) * p.N;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int64_t n = n0 + wn + j * 32 + (e >> 2) * 8 + (lane >> 5) * 4 + (e & 3);
                if (n < p.N)
                    Elem<BF16>::store(row + n, (float)acc[i][j][e] * s * bsc[n]);
            }
    }
}

}  // namespace

size_t int8_matmul_workspace(int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8_matmul(const Int8MatmulArgs &a, hipStream_t s)
{
    MatmulParams p{a.a, a.b, a.a_scale, a.b_scale, a.out, a.M, a.N, a.K, a.a_shared ? 0 : a.M, a.b_shared ? 0 : a.N,
                   (a.M + kTile - 1) / kTile, (a.N + kTile - 1) / kTile};
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * a.batch));
    if (a.bf16)
        int8_matmul_kernel<true><<<grid, dim3(256), 0, s>>>(p);
    else
        int8_matmul_kernel<false><<<grid, dim3(256), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace mamba
