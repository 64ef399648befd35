// Host side of the C ABI of the residual RMS norm, the 8-bit quantiser and the
// 8-bit matrix product: argument validation (before any HIP call) and launch.
#include "mamba_amd.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_check.h"
#include "quant.h"

namespace {

constexpr int64_t kMaxBlocks = int64_t(1) << 22;  // blocks x 1024 threads below 2^32 work-items

// Rows the token-major kernels can be launched on, with fewer than 2^32 threads:
// of up to 4096 elements four or more share a 256-thread block, wider ones have
// up to 1024 threads each.
int64_t max_rows(int64_t D) { return D <= 4096 ? (kMaxBlocks * 4 - 1) * 4 : kMaxBlocks - 1; }

// Checks of both forward norms.  `out_bytes`: of one element of `out`.
mamba_status norm_entry(const void *x, const void *residual, const float *weight, void *out, float *scale,
                        bool int8, void *residual_out, int64_t M, int64_t D, float eps, mamba_dtype io,
                        mamba_dtype residual_type, void *stream)
{
    if (!valid_dtype(io) || (residual && !valid_dtype(residual_type)))
        return MAMBA_ERR_DTYPE;
    if (!sizes_ok(M, D, 1) || !(eps >= 0.f) || std::isinf(eps))
        return MAMBA_ERR_SHAPE;
    if (D > mamba::kMaxNormWidth || (residual && io == MAMBA_F32 && residual_type == MAMBA_BF16) ||
        (residual_out && !residual))
        return MAMBA_ERR_UNSUPPORTED;
    if (M > max_rows(D))
        return MAMBA_ERR_SHAPE;
    if (M * D == 0 && !(int8 && M > 0))
        return MAMBA_OK;
    if (D == 0)
        return MAMBA_ERR_SHAPE;  // rows without elements have no scale
    if (!x || !weight || !out || (int8 && !scale))
        return MAMBA_ERR_NULL;
    const size_t es = esize(io), rs = residual ? esize(residual_type) : 0, os = int8 ? 1 : es;
    if (!aligned(x, es) || !aligned(weight, 4) || !aligned(out, os) || !aligned(scale, 4) ||
        (residual && (!aligned(residual, rs) || !aligned(residual_out, rs))))
        return MAMBA_ERR_ALIGN;
    const size_t n = (size_t)(M * D);
    const Range rx = rng(x, n * es), rr = rng(residual, n * rs), rw = rng(weight, (size_t)D * 4);
    const Range ro = rng(out, n * os), rro = rng(residual_out, residual_out ? n * rs : 0),
                rsc = rng(scale, scale ? (size_t)M * 4 : 0);
    const Range outs[] = {ro, rro, rsc};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], rx) || overlap(outs[i], rw))
            return MAMBA_ERR_ALIAS;
        // the residual may be updated in place, as the very same buffer
        const bool in_place = i == 1 && residual_out == residual;
        if (!in_place && overlap(outs[i], rr))
            return MAMBA_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], outs[j]))
                return MAMBA_ERR_ALIAS;
    }
    mamba_status st = device_ok();
    if (st != MAMBA_OK)
        return st;
    mamba::NormArgs a{x, residual, weight, out, int8 ? scale : nullptr, residual_out, M, (int)D, eps,
                      io == MAMBA_BF16, residual && residual_type == MAMBA_BF16};
    return launched(mamba::launch_rms_norm(a, (hipStream_t)stream));
}

constexpr unsigned kMatmulFlags = MAMBA_INT8_SHARED_A | MAMBA_INT8_SHARED_B;

mamba_status matmul_sizes(int64_t batch, int64_t M, int64_t N, int64_t K, unsigned flags)
{
    const bool a_shared = (flags & MAMBA_INT8_SHARED_A) != 0, b_shared = (flags & MAMBA_INT8_SHARED_B) != 0;
    if (!sizes_ok(batch, M, N) || !sizes_ok(a_shared ? 1 : batch, M, K) || !sizes_ok(b_shared ? 1 : batch, N, K))
        return MAMBA_ERR_SHAPE;
    if (K > mamba::kMaxInner || (flags & ~kMatmulFlags) != 0)
        return MAMBA_ERR_UNSUPPORTED;
    // The kernels number a batch's tiles, of 128 x 64 outputs at least where there
    // are many, in 32 bits, twice a row of them included.  Workgroups go from tile
    // to tile, so the launch itself sets no limit.
    const int64_t rows = b_shared && !a_shared ? batch * M : M;  // batches of one right operand are one
    return (rows + 127) / 128 * ((N + 63) / 64) < int64_t(1) << 30 ? MAMBA_OK : MAMBA_ERR_SHAPE;
}

}  // namespace

extern "C" {

mamba_status mamba_rms_norm(const void *x, const void *residual, const float *weight, void *out,
                            void *residual_out, int64_t M, int64_t D, float eps, mamba_dtype io,
                            mamba_dtype residual_type, void *stream)
{
    return norm_entry(x, residual, weight, out, nullptr, false, residual_out, M, D, eps, io, residual_type, stream);
}

mamba_status mamba_rms_norm_int8(const void *x, const void *residual, const float *weight, int8_t *out,
                                 float *scale, void *residual_out, int64_t M, int64_t D, float eps,
                                 mamba_dtype io, mamba_dtype residual_type, void *stream)
{
    return norm_entry(x, residual, weight, out, scale, true, residual_out, M, D, eps, io, residual_type, stream);
}

size_t mamba_rms_norm_bwd_workspace_size(int64_t M, int64_t D)
{
    if (!sizes_ok(M, D, 1) || D > mamba::kMaxNormWidth || M * D == 0)
        return 0;
    return (size_t)(mamba::rms_norm_bwd_groups(M, D) * D) * 4;
}

mamba_status mamba_rms_norm_bwd(const void *dy, const void *h, const float *weight, const void *dresidual_out,
                                void *dx, void *dresidual, float *dweight, void *workspace,
                                size_t workspace_bytes, int64_t M, int64_t D, float eps, mamba_dtype io,
                                mamba_dtype h_type, void *stream)
{
    if (!valid_dtype(io) || !valid_dtype(h_type))
        return MAMBA_ERR_DTYPE;
    if (!sizes_ok(M, D, 1) || !(eps >= 0.f) || std::isinf(eps))
        return MAMBA_ERR_SHAPE;
    if (D > mamba::kMaxNormWidth || (io == MAMBA_F32 && h_type == MAMBA_BF16) ||
        (dresidual && h_type == io))  // of one type, dx is both gradients
        return MAMBA_ERR_UNSUPPORTED;
    if (D == 0)
        return MAMBA_OK;
    if (!dweight || (M > 0 && (!dy || !h || !weight || !dx)))
        return MAMBA_ERR_NULL;
    const size_t es = esize(io), hs = esize(h_type);
    if (!aligned(dy, es) || !aligned(dx, es) || !aligned(h, hs) || !aligned(dresidual_out, hs) ||
        !aligned(dresidual, hs) || !aligned(weight, 4) || !aligned(dweight, 4))
        return MAMBA_ERR_ALIGN;
    const size_t need = mamba_rms_norm_bwd_workspace_size(M, D);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return MAMBA_ERR_WORKSPACE;
    const size_t n = (size_t)(M * D);
    const Range ins[] = {rng(dy, n * es), rng(h, n * hs), rng(dresidual_out, dresidual_out ? n * hs : 0),
                         rng(weight, M ? (size_t)D * 4 : 0)};
    const Range outs[] = {rng(dx, n * es), rng(dresidual, dresidual ? n * hs : 0), rng(dweight, (size_t)D * 4),
                          rng(workspace, need)};
    for (size_t i = 0; i < 4; ++i) {
        for (const Range &r : ins)
            if (overlap(outs[i], r))
                return MAMBA_ERR_ALIAS;
        for (size_t j = i + 1; j < 4; ++j)
            if (overlap(outs[i], outs[j]))
                return MAMBA_ERR_ALIAS;
    }
    mamba_status st = device_ok();
    if (st != MAMBA_OK)
        return st;
    mamba::NormBwdArgs a{dy, h, dresidual_out, weight, dx, dresidual, dweight, (float *)workspace, M, (int)D, eps,
                         io == MAMBA_BF16, h_type == MAMBA_BF16};
    return launched(mamba::launch_rms_norm_bwd(a, (hipStream_t)stream));
}

mamba_status mamba_quantize_int8(const void *x, int8_t *q, float *scale, int64_t B, int64_t L, int64_t K,
                                 int channel_major, mamba_dtype io, void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    if (!sizes_ok(B, L, K))
        return MAMBA_ERR_SHAPE;
    if ((channel_major != 0 && channel_major != 1) || (!channel_major && K > mamba::kMaxNormWidth))
        return MAMBA_ERR_UNSUPPORTED;
    // channel-major: a block has 16 tokens or more; fewer only in launches of few blocks
    // and of so many channels that as many blocks would need more memory than there is
    if (channel_major ? L >= kMaxBlocks * 16 || B * ((L + 15) / 16) >= kMaxBlocks : B * L > max_rows(K))
        return MAMBA_ERR_SHAPE;
    if (B * L == 0)
        return MAMBA_OK;
    if (K == 0)
        return MAMBA_ERR_SHAPE;  // tokens without channels have no scale
    if (!x || !q || !scale)
        return MAMBA_ERR_NULL;
    const size_t es = esize(io), n = (size_t)(B * L * K);
    if (!aligned(x, es) || !aligned(scale, 4))
        return MAMBA_ERR_ALIGN;
    const Range rx = rng(x, n * es), rq = rng(q, n), rs = rng(scale, (size_t)(B * L) * 4);
    if (overlap(rx, rq) || overlap(rx, rs) || overlap(rq, rs))
        return MAMBA_ERR_ALIAS;
    mamba_status st = device_ok();
    if (st != MAMBA_OK)
        return st;
    if (channel_major && !(L == 1 && K <= mamba::kMaxNormWidth)) {  // of one token, both orders are the same
        mamba::QuantChannelArgs a{x, q, scale, B, L, K, io == MAMBA_BF16};
        return launched(mamba::launch_quantize_channel_major(a, (hipStream_t)stream));
    }
    mamba::NormArgs a{x, nullptr, nullptr, q, scale, nullptr, B * L, (int)K, 0.f, io == MAMBA_BF16, false};
    return launched(mamba::launch_rms_norm(a, (hipStream_t)stream));
}

mamba_status mamba_int8_matmul(const int8_t *a, const int8_t *b, const float *a_scale, const float *b_scale,
                               void *out, int64_t batch, int64_t M, int64_t N, int64_t K, mamba_dtype out_type,
                               unsigned flags, void *stream)
{
    if (!valid_dtype(out_type))
        return MAMBA_ERR_DTYPE;
    const mamba_status sizes = matmul_sizes(batch, M, N, K, flags);
    if (sizes != MAMBA_OK || batch * M * N == 0)
        return sizes;
    const bool a_shared = (flags & MAMBA_INT8_SHARED_A) != 0, b_shared = (flags & MAMBA_INT8_SHARED_B) != 0;
    if (!out || !a_scale || !b_scale || (K > 0 && (!a || !b)))
        return MAMBA_ERR_NULL;
    if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, esize(out_type)))
        return MAMBA_ERR_ALIGN;
    const int64_t rows_a = a_shared ? M : batch * M, rows_b = b_shared ? N : batch * N;
    const Range ro = rng(out, (size_t)(batch * M * N) * esize(out_type));
    const Range ins[] = {rng(a, (size_t)(rows_a * K)), rng(b, (size_t)(rows_b * K)),
                         rng(a_scale, (size_t)rows_a * 4), rng(b_scale, (size_t)rows_b * 4)};
    for (const Range &r : ins)
        if (overlap(ro, r))
            return MAMBA_ERR_ALIAS;
    mamba_status st = device_ok();
    if (st != MAMBA_OK)
        return st;
    mamba::Int8MatmulArgs args{a, b, a_scale, b_scale, out, batch, M, N, K,
                               a_shared, b_shared, out_type == MAMBA_BF16};
    return launched(mamba::launch_int8_matmul(args, (hipStream_t)stream));
}

mamba_status mamba_int8_matmul_form(int64_t batch, int64_t M, int64_t N, int64_t K, int aligned16, unsigned flags,
                                    int *form, int64_t *tiles, int *slots)
{
    const bool a_shared = (flags & MAMBA_INT8_SHARED_A) != 0, b_shared = (flags & MAMBA_INT8_SHARED_B) != 0;
    if (!form || !tiles || !slots)
        return MAMBA_ERR_NULL;
    const mamba_status st = matmul_sizes(batch, M, N, K, flags);
    if (st != MAMBA_OK || batch * M * N == 0) {
        *form = -1;
        *tiles = *slots = 0;
        return st;
    }
    mamba::Int8MatmulArgs args{};
    args.a = aligned16 ? nullptr : (const int8_t *)1;  // for its alignment
    args.batch = batch;
    args.M = M;
    args.N = N;
    args.K = K;
    args.a_shared = a_shared;
    args.b_shared = b_shared;
    const mamba::Int8MatmulForm f = mamba::int8_matmul_form(args);
    *form = f.form;
    *tiles = f.tiles;
    *slots = f.slots;
    return MAMBA_OK;
}

}  // extern "C"
