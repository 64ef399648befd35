// Host side of the C ABI of the microscaled 4-bit format: argument validation
// (before any HIP call) and launch.
#include "mamba_amd.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "host_check.h"
#include "mxfp4.h"

namespace {

constexpr int64_t kMaxBlocks = int64_t(1) << 24;  // of 256 threads below 2^32 work-items

size_t packed_bytes(int64_t rows, int64_t K) { return (size_t)(rows * mamba::mx_groups(K)) * mamba::kMxGroupBytes; }
size_t scale_bytes(int64_t rows, int64_t K) { return (size_t)(rows * mamba::mx_groups(K)) * mamba::kMxScales; }

// Rows of whole groups: sizes within bounds, and the launches of both directions.
mamba_status row_sizes(int64_t B, int64_t L, int64_t K)
{
    if (!sizes_ok(B, L, K))
        return MAMBA_ERR_SHAPE;
    if (K > mamba::kMaxMxInner)
        return MAMBA_ERR_UNSUPPORTED;
    const int64_t groups = mamba::mx_groups(K);
    if (!sizes_ok(B, L, groups * mamba::kMxGroup) || (B * L + 31) / 32 * groups >= kMaxBlocks)
        return MAMBA_ERR_SHAPE;
    return MAMBA_OK;
}

constexpr unsigned kFlags = MAMBA_MXFP4_SHARED_A | MAMBA_MXFP4_SHARED_B;

mamba_status matmul_sizes(int64_t batch, int64_t M, int64_t N, int64_t K, unsigned flags)
{
    const bool a_shared = (flags & MAMBA_MXFP4_SHARED_A) != 0, b_shared = (flags & MAMBA_MXFP4_SHARED_B) != 0;
    if (!sizes_ok(batch, M, N) || !sizes_ok(a_shared ? 1 : batch, M, K) || !sizes_ok(b_shared ? 1 : batch, N, K))
        return MAMBA_ERR_SHAPE;
    if (K > mamba::kMaxMxInner || (flags & ~kFlags) != 0)
        return MAMBA_ERR_UNSUPPORTED;
    const int64_t padded = mamba::mx_groups(K) * mamba::kMxGroup;
    if (!sizes_ok(a_shared ? 1 : batch, M, padded) || !sizes_ok(b_shared ? 1 : batch, N, padded))
        return MAMBA_ERR_SHAPE;
    // The kernels number a batch's tiles, of 128 x 64 outputs at least where there
    // are many, in 32 bits.
    const int64_t rows = b_shared && !a_shared ? batch * M : M;  // batches of one right operand are one
    return (rows + 127) / 128 * ((N + 63) / 64) < int64_t(1) << 30 ? MAMBA_OK : MAMBA_ERR_SHAPE;
}

}  // namespace

extern "C" {

mamba_status mamba_quantize_mxfp4(const void *x, uint8_t *q, uint8_t *scale, int64_t B, int64_t L, int64_t K,
                                  int channel_major, mamba_dtype io, void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    mamba_status st = row_sizes(B, L, K);
    if (st != MAMBA_OK)
        return st;
    if (channel_major != 0 && channel_major != 1)
        return MAMBA_ERR_UNSUPPORTED;
    const int64_t rows = B * L;
    if (channel_major && B * ((L + 63) / 64) * mamba::mx_groups(K) >= kMaxBlocks / 2)  // of 512 threads
        return MAMBA_ERR_SHAPE;
    if (rows * K == 0)
        return MAMBA_OK;
    if (!x || !q || !scale)
        return MAMBA_ERR_NULL;
    const size_t es = esize(io);
    if (!aligned(x, es) || !aligned(q, 16) || !aligned(scale, 8))
        return MAMBA_ERR_ALIGN;
    const Range rx = rng(x, (size_t)(rows * K) * es), rq = rng(q, packed_bytes(rows, K)),
                rs = rng(scale, scale_bytes(rows, K));
    if (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs))
        return MAMBA_ERR_ALIAS;
    st = device_ok();
    if (st != MAMBA_OK)
        return st;
    const mamba::MxQuantArgs a{x, q, scale, B, L, K, io == MAMBA_BF16};
    if (channel_major && L > 1)  // of one token, both orders are the same
        return launched(mamba::launch_quantize_mxfp4_channel_major(a, (hipStream_t)stream));
    return launched(mamba::launch_quantize_mxfp4(a, (hipStream_t)stream));
}

mamba_status mamba_dequantize_mxfp4(const uint8_t *q, const uint8_t *scale, void *out, int64_t rows, int64_t K,
                                    mamba_dtype io, void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    mamba_status st = row_sizes(rows, 1, K);
    if (st != MAMBA_OK || rows * K == 0)
        return st;
    if (!q || !scale || !out)
        return MAMBA_ERR_NULL;
    const size_t es = esize(io);
    if (!aligned(q, 16) || !aligned(scale, 8) || !aligned(out, es))
        return MAMBA_ERR_ALIGN;
    const Range ro = rng(out, (size_t)(rows * K) * es);
    if (overlap(ro, rng(q, packed_bytes(rows, K))) || overlap(ro, rng(scale, scale_bytes(rows, K))))
        return MAMBA_ERR_ALIAS;
    st = device_ok();
    if (st != MAMBA_OK)
        return st;
    const mamba::MxDequantArgs a{q, scale, out, rows, K, io == MAMBA_BF16};
    return launched(mamba::launch_dequantize_mxfp4(a, (hipStream_t)stream));
}

mamba_status mamba_mxfp4_matmul(const uint8_t *a, const uint8_t *b, const uint8_t *a_scale, const uint8_t *b_scale,
                                void *out, int64_t batch, int64_t M, int64_t N, int64_t K, mamba_dtype out_type,
                                unsigned flags, void *stream)
{
    if (!valid_dtype(out_type))
        return MAMBA_ERR_DTYPE;
    const mamba_status sizes = matmul_sizes(batch, M, N, K, flags);
    if (sizes != MAMBA_OK || batch * M * N == 0)
        return sizes;
    const bool a_shared = (flags & MAMBA_MXFP4_SHARED_A) != 0, b_shared = (flags & MAMBA_MXFP4_SHARED_B) != 0;
    if (!out || (K > 0 && (!a || !b || !a_scale || !b_scale)))
        return MAMBA_ERR_NULL;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 8) || !aligned(b_scale, 8) ||
        !aligned(out, esize(out_type)))
        return MAMBA_ERR_ALIGN;
    const int64_t rows_a = a_shared ? M : batch * M, rows_b = b_shared ? N : batch * N;
    const Range ro = rng(out, (size_t)(batch * M * N) * esize(out_type));
    const Range ins[] = {rng(a, packed_bytes(rows_a, K)), rng(b, packed_bytes(rows_b, K)),
                         rng(a_scale, scale_bytes(rows_a, K)), rng(b_scale, scale_bytes(rows_b, K))};
    for (const Range &r : ins)
        if (overlap(ro, r))
            return MAMBA_ERR_ALIAS;
    mamba_status st = device_ok();
    if (st != MAMBA_OK)
        return st;
    const mamba::MxMatmulArgs args{a, a_scale, b, b_scale, out, batch, M, N, mamba::mx_groups(K),
                                   a_shared, b_shared, out_type == MAMBA_BF16};
    return launched(mamba::launch_mxfp4_matmul(args, (hipStream_t)stream));
}

mamba_status mamba_mxfp4_matmul_form(int64_t batch, int64_t M, int64_t N, int64_t K, unsigned flags, int *form,
                                     int64_t *tiles, int *slots)
{
    if (!form || !tiles || !slots)
        return MAMBA_ERR_NULL;
    const mamba_status st = matmul_sizes(batch, M, N, K, flags);
    if (st != MAMBA_OK || batch * M * N == 0 || K == 0) {
        *form = -1;
        *tiles = *slots = 0;
        return st;
    }
    mamba::MxMatmulArgs args{};
    args.batch = batch;
    args.M = M;
    args.N = N;
    args.groups = mamba::mx_groups(K);
    args.a_shared = (flags & MAMBA_MXFP4_SHARED_A) != 0;
    args.b_shared = (flags & MAMBA_MXFP4_SHARED_B) != 0;
    const mamba::MxMatmulForm f = mamba::mxfp4_matmul_form(args);
    *form = f.form;
    *tiles = f.tiles;
    *slots = f.slots;
    return MAMBA_OK;
}

}  // extern "C"
