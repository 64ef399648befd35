// Matrix product of microscaled 4-bit operands:
//   out[m, n] = sum over blocks of 2^(ea[m] + eb[n]) sum_k a[m, k] b[n, k]
// by the matrix cores' scaled instructions, which take a power of two for each row's
// 32 elements beside them; sums in fp32, rounded once to the output type.
//
// A wave has 32 x 32 outputs and reads its operands from memory as it goes: lane
// l % 32 a row, l / 32 one of two blocks.
#include <hip/hip_runtime.h>

#include "device_common.h"
#include "mxfp4.h"

namespace mamba {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ i32x8 wide(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <bool BF16> __global__ __launch_bounds__(256) void simple_kernel(const MxMatmulArgs p, int64_t tiles_n)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int64_t tiles_m = (p.M + 31) / 32;
    const int64_t batch = blockIdx.x / (tiles_m * tiles_n), rest = blockIdx.x % (tiles_m * tiles_n);
    const int64_t m0 = rest / tiles_n * 32, n0 = (rest % tiles_n * 4 + wave) * 32;
    const int64_t rows_a = (p.a_shared ? 1 : p.batch) * p.M, rows_b = (p.b_shared ? 1 : p.batch) * p.N;
    const int64_t m = m0 + (lane & 31), n = n0 + (lane & 31);
    const int64_t ra = (p.a_shared ? 0 : batch * p.M) + (m < p.M ? m : p.M - 1);
    const int64_t rb = (p.b_shared ? 0 : batch * p.N) + (n < p.N ? n : p.N - 1);
    const uint8_t *a = p.a + ra * p.groups * kMxGroupBytes + half * 16, *b = p.b + rb * p.groups * kMxGroupBytes + half * 16;
    f32x16 acc = {0};
    for (int64_t g = 0; g < p.groups; ++g) {
        const u32x2 sa = *(const u32x2 *)(p.a_scale + (g * rows_a + ra) * kMxScales);
        const u32x2 sb = *(const u32x2 *)(p.b_scale + (g * rows_b + rb) * kMxScales);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const i32x8 va = wide(*(const i32x4 *)(a + g * kMxGroupBytes + r * 32));
            const i32x8 vb = wide(*(const i32x4 *)(b + g * kMxGroupBytes + r * 32));
            const int ea = sa[r >> 1] >> (8 * half), eb = sb[r >> 1] >> (8 * half);
            if (r & 1)
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, acc, 4, 4, 2, eb, 2, ea);
            else
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, acc, 4, 4, 0, eb, 0, ea);
        }
    }
    if (m >= p.M)
        return;
    using T = typename Elem<BF16>::T;
    T *o = (T *)p.out + (batch * p.M + m) * p.N + n0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const int c = (q / 4) * 8 + half * 4 + q % 4;
        if (n0 + c < p.N)
            Elem<BF16>::store(o + c, acc[q]);
    }
}

}  // namespace

hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, hipStream_t s)
{
    const int64_t tiles_n = (a.N + 127) / 128;
    const dim3 grid((unsigned)(a.batch * ((a.M + 31) / 32) * tiles_n)), block(256);
    if (a.bf16)
        simple_kernel<true><<<grid, block, 0, s>>>(a, tiles_n);
    else
        simple_kernel<false><<<grid, block, 0, s>>>(a, tiles_n);
    return hipGetLastError();
}

}  // namespace mamba
