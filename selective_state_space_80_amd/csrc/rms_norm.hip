// Root-mean-square norm with the residual's addition, its 8-bit output, and
// the 8-bit quantisation of rows.
//
// Forward, per row of D elements (all in fp32):
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r w
//   residual_out = h rounded to the residual's type
//   out = y rounded to x's type, or   scale = max|y| / 127,  q = rne(y * 127 / max|y|).
// y is formed from the unrounded h: the only roundings are the outputs'.
// Where the sum of squares leaves the fp32 range (large rows; small ones without
// eps), h is taken by a power of two and summed again (range_factor).
//
// Every element is read once and written once: a row stays in the registers of
// the lanes that loaded it (8-element chunks, 16 or 32 bytes a lane), the row's
// sum (and largest value) crosses lanes by DPP and waves through LDS.
//
// Bound by memory: 16384 x 768 in fp32 with an fp32 residual (201 MB) takes
// 39 us (5.1 TB/s, the rate of a large copy); 16384 x 2560 bf16 with a bf16
// residual 60 us, with 8-bit output 54 us (5.6 and 5.4 TB/s); 131072 rows of 64
// bf16 6.7 us from the last-level cache (with a wave to each row, more than
// twice that).  One row of 2560 is bound by its launch.
#include <hip/hip_runtime.h>

#include "quant.h"
#include "row_chunk.h"

namespace mamba {
namespace {

enum Mode { kNorm, kNormInt8, kQuant };

struct NormParams {
    const void *x, *res;
    const float *w;
    void *out;
    float *scale;
    void *res_out;
    int64_t M;
    int D;
    float eps, inv_d;
};

// RES: 0 no residual, 1 fp32, 2 bf16.  LANES > 0: every LANES lanes of a
// workgroup's four waves have a row of their own; 0: the workgroup (any number
// of waves) has one row.  NC chunks a lane.
template <bool XBF, int RES, int MODE, int LANES, int NC, bool TINY>
__global__ __launch_bounds__(LANES ? 256 : 1024) void rms_norm_kernel(const NormParams p)
{
    using XT = typename Elem<XBF>::T;
    using RT = typename Elem<RES == 2>::T;
    __shared__ float red[3][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRows = LANES ? 64 / LANES : 1;  // of a wave
    const int n_waves = LANES ? 1 : (int)(blockDim.x >> 6);
    int64_t row = LANES ? ((int64_t)blockIdx.x * 4 + wave) * kRows : (int64_t)blockIdx.x;
    if (LANES && row >= p.M)
        return;  // the whole wave; no barrier follows in this form
    bool past = false;  // lanes of rows past the last repeat it and store nothing
    if constexpr (kRows > 1) {
        row += lane / LANES;
        past = row >= p.M;
        row = past ? p.M - 1 : row;
    }
    const int tid = LANES ? lane % LANES : (int)threadIdx.x;
    const int T = LANES ? LANES : (int)blockDim.x;
    const int D = p.D;
    const bool ragged = D % kChunk != 0;

    ChunkAt at[NC];
    float h[NC][8];
    const XT *xr = (const XT *)p.x + row * D;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        at[j] = chunk_at<TINY>(tid + j * T, D);
        if (past)
            at[j].live = false;
        load_chunk<XBF, TINY>(xr, at[j], D, h[j]);
    }
    if constexpr (RES != 0) {
        const RT *rr = (const RT *)p.res + row * D;
        float r[NC][8];
#pragma unroll
        for (int j = 0; j < NC; ++j)
            load_chunk<RES == 2, TINY>(rr, at[j], D, r[j]);
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[j][i] += r[j][i];
    }
    if constexpr (MODE != kQuant) {
        float w[NC][8];
#pragma unroll
        for (int j = 0; j < NC; ++j)
            load_chunk<false, TINY>(p.w, at[j], D, w[j]);
        auto square_sum = [&](float(&slots)[16]) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < NC; ++j)
                s += own_sum<TINY>(at[j], D, ragged, [&](int i) { return h[j][i] * h[j][i]; });
            s = lane_sum<LANES ? LANES : 64>(s);
            if constexpr (!LANES) {
                if (lane == 0)
                    slots[wave] = s;
                __syncthreads();
                s = slots[0];
                for (int k = 1; k < n_waves; ++k)
                    s += slots[k];
            }
            return s;
        };
        float s = square_sum(red[0]), eps = p.eps;
        // every element of the row has been read: the residual may be overwritten
        if constexpr (RES != 0) {
            if (p.res_out) {
                RT *ro = (RT *)p.res_out + row * D;
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    store_chunk<RES == 2, TINY>(ro, at[j], D, h[j]);
            }
        }
        const float factor = range_factor(s, eps);  // the same in all lanes of the row
        if (__builtin_expect(factor != 1.f, 0)) {
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[j][i] *= factor;
            s = square_sum(red[2]);
            eps = eps * factor * factor;
            if (s == 0.f && eps == 0.f)
                eps = 1.f;  // a zero row stays zero
        }
        const float r = inv_root(fmaf(s, p.inv_d, eps));
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                h[j][i] = h[j][i] * r * w[j][i];
    }
    if constexpr (MODE == kNorm) {
        XT *yo = (XT *)p.out + row * D;
#pragma unroll
        for (int j = 0; j < NC; ++j)
            store_chunk<XBF, TINY>(yo, at[j], D, h[j]);
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)  // lanes without a chunk hold the row's first: no mask
                top = umax(top, abs_bits(h[j][i]));
        top = lane_max<LANES ? LANES : 64>(top);
        if constexpr (!LANES) {
            if (lane == 0)
                red[1][wave] = __uint_as_float(top);
            __syncthreads();
            for (int k = 0; k < n_waves; ++k)
                top = umax(top, __float_as_uint(red[1][k]));
        }
        const RowScale<XBF && MODE == kQuant> rs(top);  // the norm's values are fp32
        if (tid == 0 && !past)
            p.scale[row] = rs.scale;
        if (rs.raise != 1.f) {
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    h[j][i] *= rs.raise;
        }
        int8_t *qo = (int8_t *)p.out + row * D;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const u32x2 q = pack_int8(h[j], rs);
            if (!at[j].live)
                continue;
            if constexpr (TINY) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < D)
                        qo[i] = (int8_t)(q[i / 4] >> (8 * (i % 4)));
            } else {
                __builtin_memcpy(qo + at[j].off, &q, 8);
            }
        }
    }
}

template <bool XBF, int RES, int MODE, int LANES, int NC, bool TINY>
hipError_t start(const NormParams &p, int threads, hipStream_t s)
{
    constexpr int kRows = LANES ? 4 * (64 / LANES) : 1;
    const int64_t blocks = (p.M + kRows - 1) / kRows;
    rms_norm_kernel<XBF, RES, MODE, LANES, NC, TINY><<<dim3((unsigned)blocks), dim3(threads), 0, s>>>(p);
    return hipGetLastError();
}

template <bool XBF, int RES, int MODE> hipError_t pick(const NormParams &p, hipStream_t s)
{
    if (p.D < kChunk)
        return start<XBF, RES, MODE, 8, 1, true>(p, 256, s);
    switch (row_lanes(p.D)) {
    case 8: return start<XBF, RES, MODE, 8, 1, false>(p, 256, s);
    case 16: return start<XBF, RES, MODE, 16, 1, false>(p, 256, s);
    case 32: return start<XBF, RES, MODE, 32, 1, false>(p, 256, s);
    }
    // A wave holds up to 8 chunks a lane (4096 elements); with fewer rows than
    // fill the card with waves, a workgroup shares a row instead.  Both sides, a
    // workgroup to a row and a wave, bf16 with 8-bit output in us: 256 x 2560 3.4 and
    // 3.9, 512 4.3 and 4.4, 768 5.1 and 5.0, 1024 5.8 and 5.6, 2048 10.4 and 9.5.  The
    // bound is a compromise: 768 elements cross at 256 rows (2048 x 768 4.5 and
    // 4.3), 4096 not up to 4096 rows (1024 x 4096 7.6 and 8.3), nor does fp32
    // (1024 x 2560 10.9 and 11.1, 4096 33.8 and 35.5).
    const int chunks = (p.D + kChunk - 1) / kChunk;
    const int per_lane = (chunks + 63) / 64;
    if (per_lane <= 1 || (per_lane <= 8 && p.M >= 1024)) {
        switch (per_lane) {
        case 1: return start<XBF, RES, MODE, 64, 1, false>(p, 256, s);
        case 2: return start<XBF, RES, MODE, 64, 2, false>(p, 256, s);
        case 3: return start<XBF, RES, MODE, 64, 3, false>(p, 256, s);
        case 4: return start<XBF, RES, MODE, 64, 4, false>(p, 256, s);
        case 5: return start<XBF, RES, MODE, 64, 5, false>(p, 256, s);
        default: return start<XBF, RES, MODE, 64, 8, false>(p, 256, s);
        }
    }
    // Of a shared row a lane takes one chunk up to 512, then two: workgroups of
    // 1024 lanes leave a CU too few rows at once (bf16 with 8-bit output, in us: 16384 x 5120 103
    // with two and 130 with one; 8192 x 8192 84 and 93).  Four only where two
    // no longer cover the row.
    const int nc = chunks <= 512 ? 1 : chunks <= 2048 ? 2 : 4;
    const int lanes = (chunks + nc - 1) / nc;
    const int threads = (lanes + 63) / 64 * 64;
    if (nc == 1)
        return start<XBF, RES, MODE, 0, 1, false>(p, threads, s);
    if (nc == 2)
        return start<XBF, RES, MODE, 0, 2, false>(p, threads, s);
    return start<XBF, RES, MODE, 0, 4, false>(p, threads, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s)
{
    NormParams p{a.x, a.residual, a.weight, a.out, a.scale, a.residual_out, a.M, a.D, a.eps, 1.f / (float)a.D};
    if (!a.weight)
        return a.bf16 ? pick<true, 0, kQuant>(p, s) : pick<false, 0, kQuant>(p, s);
    const int res = !a.residual ? 0 : a.residual_bf16 ? 2 : 1;
    if (a.scale) {
        if (!a.bf16)
            return res ? pick<false, 1, kNormInt8>(p, s) : pick<false, 0, kNormInt8>(p, s);
        return res == 2 ? pick<true, 2, kNormInt8>(p, s)
               : res    ? pick<true, 1, kNormInt8>(p, s)
                        : pick<true, 0, kNormInt8>(p, s);
    }
    if (!a.bf16)
        return res ? pick<false, 1, kNorm>(p, s) : pick<false, 0, kNorm>(p, s);
    return res == 2 ? pick<true, 2, kNorm>(p, s)
           : res    ? pick<true, 1, kNorm>(p, s)
                    : pick<true, 0, kNorm>(p, s);
}

}  // namespace mamba
