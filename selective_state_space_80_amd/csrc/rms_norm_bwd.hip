// Gradient of the root-mean-square norm with the residual's addition.
//
// With h the stored sum, r = 1 / sqrt(mean(h^2) + eps) and y = h r w:
//   dh = r (w dy) - h r^3 mean(w dy h) + dres_out      (dx, and the residual's gradient)
//   dw = sum over rows of dy h r
// Both row sums (h^2 and w dy h) need no r, so one pass over the row gives
// them together; dh follows from the registers.  dw is summed over the rows a
// workgroup takes in its registers, written once per workgroup, and summed
// over the workgroups in a fixed order by a second kernel.
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
// DRES: dres_out is given.  WAVE_ROW as in the forward kernel.
template <bool XBF, bool HF32, bool DRES, bool WAVE_ROW, int NC, bool TINY>
__global__ __launch_bounds__(WAVE_ROW ? 256 : NC == 1 ? 512 : 1024) void rms_norm_bwd_kernel(const BwdParams p)
{
    constexpr bool HBF = XBF && !HF32;
    using XT = typename Elem<XBF>::T;
    using HT = typename Elem<HBF>::T;
    __shared__ float red[2][2][16];
    __shared__ float dw_red[WAVE_ROW ? 4 : 1][WAVE_ROW ? NC * 512 : 1];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n_waves = WAVE_ROW ? 1 : (int)(blockDim.x >> 6);
    const int tid = WAVE_ROW ? lane : (int)threadIdx.x;
    const int T = WAVE_ROW ? 64 : (int)blockDim.x;
    const int D = p.D;
    const bool ragged = D % kChunk != 0;
    const int64_t step = WAVE_ROW ? (int64_t)gridDim.x * 4 : (int64_t)gridDim.x;
    const int64_t first = WAVE_ROW ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;

    ChunkAt at[NC];
    float w[NC][8], acc[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        at[j] = chunk_at<TINY>(tid + j * T, D);
        load_chunk<false, TINY>(p.w, at[j], D, w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[j][i] = 0.f;
    }
    // Where registers allow, the next row is loaded while this one is worked on
    // (PERF).
    constexpr bool kAhead = WAVE_ROW || NC == 1;
    RawChunk<HBF> rh[NC], rd[NC];
    RawChunk<XBF> rg[NC];
    auto load_row = [&](int64_t row) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            rh[j].template load<TINY>((const HT *)p.h + row * D, at[j], D);
            rg[j].template load<TINY>((const XT *)p.dy + row * D, at[j], D);
            if constexpr (DRES)
                rd[j].template load<TINY>((const HT *)p.dres_out + row * D, at[j], D);
        }
    };
    if (kAhead && first < p.M)
        load_row(first);
    int parity = 0;
    for (int64_t row = first; row < p.M; row += step) {
        if (!kAhead)
            load_row(row);
        float h[NC][8], g[NC][8], d[NC][8];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            rh[j].get(h[j]);
            rg[j].get(g[j]);
            if constexpr (DRES)
                rd[j].get(d[j]);
        }
        if (kAhead && row + step < p.M)
            load_row(row + step);
        float s = 0.f, t = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            s += own_sum<TINY>(at[j], D, ragged, [&](int i) { return h[j][i] * h[j][i]; });
            t += own_sum<TINY>(at[j], D, ragged, [&](int i) { return g[j][i] * w[j][i] * h[j][i]; });
        }
        s = wave_sum(s);
        t = wave_sum(t);
        if constexpr (!WAVE_ROW) {
            // two sets of slots in turn: a wave writes the next row's while
            // others still read this row's
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
        const float r = 1.f / sqrtf(fmaf(s, p.inv_d, p.eps));
        const float k3 = r * r * r * (t * p.inv_d);
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float dh[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[j][i] = fmaf(g[j][i] * r, h[j][i], acc[j][i]);
                dh[i] = fmaf(r * w[j][i], g[j][i], -k3 * h[j][i]);
                if constexpr (DRES)
                    dh[i] += d[j][i];
            }
            store_chunk<XBF, TINY>((XT *)p.dx + row * D, at[j], D, dh);
            if constexpr (HF32) {
                if (p.dres)
                    store_chunk<false, TINY>((float *)p.dres + row * D, at[j], D, dh);
            }
        }
    }
    float *part = p.partials + (int64_t)blockIdx.x * D;
    const int end = TINY ? D : kChunk;
    if constexpr (WAVE_ROW) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dw_red[wave][(j * 64 + lane) * 8 + i] = acc[j][i];
        __syncthreads();
        if (wave != 0)
            return;
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = (j * 64 + lane) * 8 + i;
                acc[j][i] = ((dw_red[0][k] + dw_red[1][k]) + dw_red[2][k]) + dw_red[3][k];
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

// Workgroups: enough of them to fill 256 CUs, at least 8 rows each where there
// are so many, so that the partial rows stay a small part of the traffic.
constexpr int64_t kMaxGroups = 1024;

bool wave_row(int64_t D) { return D <= 1024; }

template <bool XBF, bool HF32, bool DRES, bool WAVE_ROW, int NC, bool TINY>
hipError_t start(const BwdParams &p, int64_t groups, int threads, hipStream_t s)
{
    rms_norm_bwd_kernel<XBF, HF32, DRES, WAVE_ROW, NC, TINY>
        <<<dim3((unsigned)groups), dim3(threads), 0, s>>>(p);
    return hipGetLastError();
}

template <bool XBF, bool HF32, bool DRES> hipError_t pick(const BwdParams &p, int64_t groups, hipStream_t s)
{
    if (p.D < kChunk)
        return start<XBF, HF32, DRES, true, 1, true>(p, groups, 256, s);
    const int chunks = (p.D + kChunk - 1) / kChunk;
    if (wave_row(p.D))
        return chunks <= 64 ? start<XBF, HF32, DRES, true, 1, false>(p, groups, 256, s)
                            : start<XBF, HF32, DRES, true, 2, false>(p, groups, 256, s);
    const int nc = chunks <= 512 ? 1 : chunks <= 2048 ? 2 : 4;
    const int lanes = (chunks + nc - 1) / nc;
    const int threads = (lanes + 63) / 64 * 64;
    if (nc == 1)
        return start<XBF, HF32, DRES, false, 1, false>(p, groups, threads, s);
    if (nc == 2)
        return start<XBF, HF32, DRES, false, 2, false>(p, groups, threads, s);
    return start<XBF, HF32, DRES, false, 4, false>(p, groups, threads, s);
}

}  // namespace

int64_t rms_norm_bwd_groups(int64_t M, int64_t D)
{
    const int64_t rows_at_once = wave_row(D) ? 4 : 1;
    const int64_t most = (M + rows_at_once - 1) / rows_at_once;
    const int64_t wanted = most < 256 ? most : (most / 8 > 256 ? most / 8 : 256);
    return wanted < kMaxGroups ? wanted : kMaxGroups;
}

hipError_t launch_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s)
{
    const int64_t groups = rms_norm_bwd_groups(a.M, a.D);
    if (groups > 0) {
        BwdParams p{a.dy, a.h, a.dres_out, a.weight, a.dx, a.dres, a.partials, a.M, a.D, a.eps, 1.f / (float)a.D};
        hipError_t e;
        if (!a.bf16)
            e = a.dres_out ? pick<false, false, true>(p, groups, s) : pick<false, false, false>(p, groups, s);
        else if (a.h_bf16)
            e = a.dres_out ? pick<true, false, true>(p, groups, s) : pick<true, false, false>(p, groups, s);
        else
            e = a.dres_out ? pick<true, true, true>(p, groups, s) : pick<true, true, false>(p, groups, s);
        if (e != hipSuccess)
            return e;
    }
    dweight_sum_kernel<<<dim3((unsigned)((a.D + 31) / 32)), dim3(1024), 0, s>>>(a.partials, a.dweight, groups, a.D);
    return hipGetLastError();
}

}  // namespace mamba
