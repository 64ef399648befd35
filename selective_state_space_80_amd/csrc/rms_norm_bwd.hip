// Gradient of the root-mean-square norm with the residual's addition.
//
// With h the stored sum, r = 1 / sqrt(mean(h^2) + eps) and y = h r w:
//   dh = r (w dy - (h r) r mean(w dy h)) + dres_out      (dx, and the residual's gradient)
//   dw = sum over rows of dy h r
// Both row sums (h^2 and w dy h) need no r, so one pass over the row gives
// them together; dh follows from the registers.  dw is summed over the rows a
// workgroup takes in its registers, written once per workgroup, and summed
// over the workgroups in a fixed order by a second kernel.  Rows whose sum of
// squares leaves the fp32 range are taken by a power of two, as in the forward
// kernel.
//
// Bound by memory: 16384 x 2560, dy and dx bf16, h and both residual gradients
// fp32 (671 MB), takes 129 us (5.2 TB/s, the rate of a large copy);
// 16384 x 768 in fp32 (201 MB) 38 us; 1044 x 2339 is bound by its two launches.
#include <hip/hip_runtime.h>

#include "quant.h"
#include "row_chunk.h"

namespace mamba {
namespace {

struct BwdParams {
    const void *dy, *h, *dres_out;
    const float *w;
    void *dx, *dres;
    float *partials;
    int64_t M;
    int D;
    float eps, inv_d;
};

// HF32: h (and the residual gradients) are fp32 while dy and dx are bf16.
// DRES: dres_out is given.  LANES as in the forward kernel.
template <bool XBF, bool HF32, bool DRES, int LANES, int NC, bool TINY>
__global__ __launch_bounds__(LANES ? 256 : NC == 1 ? 512 : 1024) void rms_norm_bwd_kernel(const BwdParams p)
{
    constexpr bool HBF = XBF && !HF32;
    using XT = typename Elem<XBF>::T;
    using HT = typename Elem<HBF>::T;
    __shared__ float red[2][2][16];
    __shared__ float dw_red[LANES ? 4 : 1][LANES ? NC * 512 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRows = LANES ? 64 / LANES : 1;  // of a wave
    const int n_waves = LANES ? 1 : (int)(blockDim.x >> 6);
    const int tid = LANES ? lane % LANES : (int)threadIdx.x;
    const int T = LANES ? LANES : (int)blockDim.x;
    const int D = p.D;
    const bool ragged = D % kChunk != 0;
    const int64_t step = LANES ? (int64_t)gridDim.x * 4 * kRows : (int64_t)gridDim.x;
    const int64_t first = LANES ? ((int64_t)blockIdx.x * 4 + wave) * kRows : (int64_t)blockIdx.x;
    const int sub = kRows > 1 ? lane / LANES : 0;  // its row of the wave's

    ChunkAt at[NC];
    // Four chunks a lane leave no registers for the weight, which is then read
    // again for each row, nor for dres_out before it is needed (2048 x 20000,
    // bf16 with fp32 h: 159 us; with all of it in registers, spilling, 259).  Some
    // values are spilled all the same, 11 or 12 in fp32 and up to 3 in bf16 (2048 x
    // 20000 in fp32 168 us; 172 when 46 were).
    constexpr bool kLean = NC == 4;
    float w[kLean ? 1 : NC][8], acc[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        at[j] = chunk_at<TINY>(tid + j * T, D);
        if constexpr (!kLean)
            load_chunk<false, TINY>(p.w, at[j], D, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[j][i] = 0.f;
    }
    // Where registers allow, the next row is loaded while this one is worked on.
    constexpr bool kAhead = LANES != 0 || NC == 1;
    RawChunk<HBF> rh[NC], rd[kLean ? 1 : NC];
    RawChunk<XBF> rg[NC];
    auto load_row = [&](int64_t row) {
        if constexpr (kRows > 1)  // lanes of rows past the last repeat it
            row = row + sub < p.M ? row + sub : p.M - 1;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            rh[j].template load<TINY>((const HT *)p.h + row * D, at[j], D);
            rg[j].template load<TINY>((const XT *)p.dy + row * D, at[j], D);
            if constexpr (DRES && !kLean)
                rd[j].template load<TINY>((const HT *)p.dres_out + row * D, at[j], D);
        }
    };
    if (kAhead && first < p.M)
        load_row(first);
    int parity = 0;
    for (int64_t row = first; row < p.M; row += step) {
        if (!kAhead)
            load_row(row);
        float h[kLean ? 1 : NC][8], g[kLean ? 1 : NC][8], d[kLean ? 1 : NC][8];
        if constexpr (!kLean) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                rh[j].get(h[j]);
                rg[j].get(g[j]);
                if constexpr (DRES && kAhead)
                    rd[j].get(d[j]);
            }
        }
        // What a lean lane needs of chunk j.  The empty statement keeps the
        // compiler from carrying the results of one use to the next in registers.
        const float *weight = p.w;
        auto unpack = [&](int j, float factor) {
            if constexpr (kLean) {
                asm volatile("" : "+s"(weight));
                rh[j].keep();
                rg[j].keep();
                rh[j].get(h[0]);
                rg[j].get(g[0]);
                if (__builtin_expect(factor != 1.f, 0)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        h[0][i] *= factor;
                }
                load_chunk<false, TINY>(weight, at[j], D, w[0]);
            }
        };
        if (kAhead && row + step < p.M)
            load_row(row + step);
        float s, t, factor = 1.f, eps = p.eps;
        auto sums = [&]() {
            s = t = 0.f;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int k = kLean ? 0 : j;
                unpack(j, factor);
                s += own_sum<TINY>(at[j], D, ragged, [&](int i) { return h[k][i] * h[k][i]; });
                t += own_sum<TINY>(at[j], D, ragged, [&](int i) { return g[k][i] * w[k][i] * h[k][i]; });
            }
            s = lane_sum<LANES ? LANES : 64>(s);
            t = lane_sum<LANES ? LANES : 64>(t);
            if constexpr (!LANES) {
                // two sets of slots in turn: a wave writes the next sums while
                // others still read these
                if (lane == 0) {
                    red[parity][0][wave] = s;
                    red[parity][1][wave] = t;
                }
                __syncthreads();
                s = red[parity][0][0];
                t = red[parity][1][0];
                for (int k = 1; k < n_waves; ++k) {
                    s += red[parity][0][k];
                    t += red[parity][1][k];
                }
                parity ^= 1;
            }
        };
        auto zero_row = [&]() {  // without eps: no gradient through the norm
            if (s == 0.f && eps == 0.f) {
                eps = 1.f;
                factor = 0.f;
            }
        };
        // Rows whose square sum leaves the fp32 range take a second pass.  Lean
        // lanes loop, so that the registers are laid out for one (fp32: 12 spilled, 50 with two).
        if constexpr (kLean) {
#pragma unroll 1
            for (;;) {
                sums();
                if (__builtin_expect(factor != 1.f, 0)) {
                    zero_row();
                    break;
                }
                factor = range_factor(s, eps);  // the same in all lanes of the row
                if (__builtin_expect(factor == 1.f, 1))
                    break;
                eps = eps * factor * factor;
            }
        } else {
            sums();
            factor = range_factor(s, eps);
            if (__builtin_expect(factor != 1.f, 0)) {
                eps = eps * factor * factor;
#pragma unroll
                for (int j = 0; j < NC; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        h[j][i] *= factor;
                sums();
                zero_row();
            }
        }
        // of the elements with the factor, and of the row itself
        const float r = inv_root(fmaf(s, p.inv_d, eps)), row_r = r * factor;
        const float c = t * r * p.inv_d;
        if constexpr (DRES && !kAhead && !kLean) {  // the last loads are waited for before the first store
#pragma unroll
            for (int j = 0; j < NC; ++j)
                rd[j].keep();
        }
        const bool past = kRows > 1 && row + sub >= p.M;
        const int64_t mine = kRows > 1 ? row + sub : row;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            if (past)
                continue;
            const int k = kLean ? 0 : j;
            unpack(j, factor);
            if constexpr (kLean && DRES)
                load_chunk<HBF, TINY>((const HT *)p.dres_out + mine * D, at[j], D, d[0]);
            if constexpr (!kLean && DRES && !kAhead)
                rd[j].get(d[j]);
            float dh[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float hr = h[k][i] * r;  // normalised: r^3 passes the fp32 range before it does
                acc[j][i] = fmaf(g[k][i], hr, acc[j][i]);
                dh[i] = row_r * fmaf(g[k][i], w[k][i], -c * hr);
                if constexpr (DRES)
                    dh[i] += d[k][i];
            }
            store_chunk<XBF, TINY>((XT *)p.dx + mine * D, at[j], D, dh);
            if constexpr (HF32) {
                if (p.dres)
                    store_chunk<false, TINY>((float *)p.dres + mine * D, at[j], D, dh);
            }
        }
    }
    float *part = p.partials + (int64_t)blockIdx.x * D;
    const int end = TINY ? D : kChunk;
    if constexpr (LANES != 0) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dw_red[wave][(j * 64 + lane) * 8 + i] = acc[j][i];
        __syncthreads();
        if (wave != 0 || sub != 0)
            return;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float sum = 0.f;
#pragma unroll
                for (int r = 0; r < 4 * kRows; ++r)
                    sum += dw_red[r / kRows][(j * 64 + r % kRows * LANES + lane) * 8 + i];
                acc[j][i] = sum;
            }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j)
        if (at[j].live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= at[j].lo && i < end)
                    part[at[j].off + i] = acc[j][i];
        }
}

// dweight[c] = sum over the groups' partial rows, 32 columns by 32 slices of
// the groups per workgroup, each slice and then the slices in order.
__global__ __launch_bounds__(1024) void dweight_sum_kernel(const float *partials, float *dweight, int64_t groups,
                                                           int D)
{
    __shared__ float part[32][33];
    const int col = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + col;
    float s = 0.f;
    if (c < D) {
        const int64_t per = (groups + 31) / 32;
        const int64_t from = slice * per, to = from + per < groups ? from + per : groups;
#pragma unroll 8
        for (int64_t g = from; g < to; ++g)
            s += partials[g * D + c];
    }
    part[slice][col] = s;
    __syncthreads();
    if (slice == 0 && c < D) {
        float sum = part[0][col];
#pragma unroll
        for (int k = 1; k < 32; ++k)
            sum += part[k][col];
        dweight[c] = sum;
    }
}

// Workgroups: at least 8 rows each where there are so many, and not more than
// the card runs at once, so that the partial rows stay a small part of the
// traffic.  Two a CU, four of the light ones of short rows: 8192 x 5120 bf16
// 48 us with 512 of them, 59 with 1024; 17929 x 567 fp32 26 and 31; but
// 131072 x 320 bf16 62 and 52.
int64_t most_groups(int64_t D) { return D <= 512 ? 1024 : 512; }

// Up to 1024 elements a wave holds whole rows.
int64_t rows_at_once(int64_t D) { return D <= 1024 ? 4 * (64 / row_lanes(D)) : 1; }

template <bool XBF, bool HF32, bool DRES, int LANES, int NC, bool TINY>
hipError_t start(const BwdParams &p, int64_t groups, int threads, hipStream_t s)
{
    rms_norm_bwd_kernel<XBF, HF32, DRES, LANES, NC, TINY>
        <<<dim3((unsigned)groups), dim3(threads), 0, s>>>(p);
    return hipGetLastError();
}

template <bool XBF, bool HF32, bool DRES> hipError_t pick(const BwdParams &p, int64_t groups, hipStream_t s)
{
    if (p.D < kChunk)
        return start<XBF, HF32, DRES, 8, 1, true>(p, groups, 256, s);
    switch (row_lanes(p.D)) {
    case 8: return start<XBF, HF32, DRES, 8, 1, false>(p, groups, 256, s);
    case 16: return start<XBF, HF32, DRES, 16, 1, false>(p, groups, 256, s);
    case 32: return start<XBF, HF32, DRES, 32, 1, false>(p, groups, 256, s);
    }
    const int chunks = (p.D + kChunk - 1) / kChunk;
    if (chunks <= 64)
        return start<XBF, HF32, DRES, 64, 1, false>(p, groups, 256, s);
    if (chunks <= 128)
        return start<XBF, HF32, DRES, 64, 2, false>(p, groups, 256, s);
    // More chunks a lane mean fewer waves with more registers and sums each, so
    // the fewest that the row allows (with dres, four sets of tensors in turn so that
    // they come from memory, in us: 16384 x 2560 67 with one and 84 with
    // two, 4096 x 10240 81 with two and 101 with four), except that rows of 513
    // to 1024 chunks take two, as in the forward pass (4096 x 8192 59 with two and
    // 61 with one; 8192 x 5120 71 and 71).
    const int nc = chunks <= 512 ? 1 : chunks <= 2048 ? 2 : 4;
    const int lanes = (chunks + nc - 1) / nc;
    const int threads = (lanes + 63) / 64 * 64;
    if (nc == 1)
        return start<XBF, HF32, DRES, 0, 1, false>(p, groups, threads, s);
    if (nc == 2)
        return start<XBF, HF32, DRES, 0, 2, false>(p, groups, threads, s);
    return start<XBF, HF32, DRES, 0, 4, false>(p, groups, threads, s);
}

}  // namespace

int64_t rms_norm_bwd_groups(int64_t M, int64_t D)
{
    const int64_t at_once = rows_at_once(D), most = (M + at_once - 1) / at_once;
    const int64_t wanted = most < 256 ? most : (most / 8 > 256 ? most / 8 : 256);
    return wanted < most_groups(D) ? wanted : most_groups(D);
}

hipError_t launch_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s)
{
    const int64_t groups = rms_norm_bwd_groups(a.M, a.D);
    if (groups > 0) {
        // a single group's partial row is the gradient itself
        float *partials = groups == 1 ? a.dweight : a.partials;
        BwdParams p{a.dy, a.h, a.dres_out, a.weight, a.dx, a.dres, partials, a.M, a.D, a.eps, 1.f / (float)a.D};
        hipError_t e;
        if (!a.bf16)
            e = a.dres_out ? pick<false, false, true>(p, groups, s) : pick<false, false, false>(p, groups, s);
        else if (a.h_bf16)
            e = a.dres_out ? pick<true, false, true>(p, groups, s) : pick<true, false, false>(p, groups, s);
        else
            e = a.dres_out ? pick<true, true, true>(p, groups, s) : pick<true, true, false>(p, groups, s);
        if (e != hipSuccess || groups == 1)
            return e;
    }
    dweight_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32)), dim3(1024), 0, s>>>(a.partials, a.dweight, groups, a.D);
    return hipGetLastError();
}

}  // namespace mamba
