// Gated linear recurrence, backward.  With g_t the gradient that reaches h_t,
//   g_t  = dout_t SiLU(z_t) + a_(t+1) g_(t+1)          (dh_last behind the last step)
//   dx_t = g m s,   di_t = g m x s (1 - s),   s = sigmoid(i)
//   dv_t = -a (g h_(t-1)) + (a^2 / m) g s x            (0 at a reset)
//   dr_t = dv v (1 - sigmoid(r)),   dlam = sum dv v sigmoid(lam) / softplus(lam)
//   dz_t = dout h SiLU'(z),   dh0 = a_0 g_0
// (m = sqrt(1 - a^2), dm/dv = a^2 / m; v / m -> 0 with v, so dv is taken with its v.)
// Rows go by as in the forward kernel, from the last chunk to the first.  The states
// come from the forward call's checkpoints, one a chunk, and the steps after it run
// again; so a chunk needs nothing from its neighbours but the gradient that enters it
// from behind, a_(t+1) g_(t+1), and the inputs are read once.  Bound by memory: 8 x 5120
// x 2048 bf16 215 us, 5.5 TB/s, gated 260 to 278.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gated_common.h"
#include "gated_scan.h"

namespace mamba {
namespace {

// sigmoid(lam) / softplus(lam), which goes to 1 where both go to 0.
__device__ __forceinline__ float lam_slope(float lam)
{
    const float t = expf(-fabsf(lam)), s = (lam < 0.f ? t : 1.f) / (1.f + t);
    return lam < -80.f ? 1.f : s / softplus_row(lam);
}

template <int G, int WAVES, bool BF16, bool GATE, bool RESET, bool PARTS>
__global__ __launch_bounds__(gated_threads(WAVES)) void gated_bwd_kernel(const GatedScanBwdArgs p)
{
    using T = typename Elem<BF16>::T;
    using M = Span<RESET>;
    constexpr int kRows = gated_threads(WAVES) / G / WAVES;  // of a workgroup
    constexpr int kSpan = G * kLaneSteps * WAVES;
    __shared__ float2 maps[2][WAVES];
    __shared__ float sums[3][WAVES];
    const int lane = threadIdx.x & (G - 1), wave = uniform<G == 64>(threadIdx.x / G % WAVES);
    const int rows = (int)(p.f.B * p.f.D), row = uniform<G == 64>(blockIdx.x * kRows + threadIdx.x / (G * WAVES));
    const bool live = row < rows;
    const int64_t start = PARTS ? blockIdx.y * p.f.part_steps : 0;
    const int64_t stop = PARTS && start + p.f.part_steps < p.f.L ? start + p.f.part_steps : p.f.L;
    const int64_t at = live ? row : 0, L = live ? stop : 0, first_of = at * p.f.L;
    const uint32_t d = (uint32_t)at % (uint32_t)p.f.D;  // rows are below 2^24
    const T *x = (const T *)p.f.x + first_of, *r = (const T *)p.f.r + first_of, *i = (const T *)p.f.i + first_of;
    const T *z = GATE ? (const T *)p.f.z + first_of : nullptr, *dout = (const T *)p.dout + first_of;
    T *dx = (T *)p.dx + first_of, *dr = (T *)p.dr + first_of, *di = (T *)p.di + first_of;
    T *dz = GATE ? (T *)p.dz + first_of : nullptr;
    const uint8_t *reset = RESET ? p.f.reset + (int64_t)((uint32_t)at / (uint32_t)p.f.D) * p.f.L : nullptr;
    const float lam = p.f.lam[d], r_bias = p.f.r_bias ? p.f.r_bias[d] : 0.f, i_bias = p.f.i_bias ? p.f.i_bias[d] : 0.f;
    const int64_t chunks = (p.f.L + kGatedChunk - 1) / kGatedChunk;
    float carry = p.dh_last ? p.dh_last[at] : 0.f;  // a g of the step behind
    if constexpr (PARTS)
        carry = through_parts<RESET>(p.f.maps + at * p.f.parts, p.f.parts - 1 - (int)blockIdx.y, true, p.f.parts, carry);
    float sum_q = 0.f, sum_r = 0.f, sum_i = 0.f;

    Eight<BF16> nx, nr, ni, nz, nd;
    uint32_t nreset = 0;
    float nstate = 0.f;
    const uint32_t off = lane * kLaneSteps;
    auto fetch = [&](int64_t t) {
        const int left = steps_left<G>(L, t), n = lane_share(left, off);
        const bool whole = G == 64 && left == G * kLaneSteps;
        load_some<BF16>(nr, r + t + off, whole, n, -__builtin_inff());  // past the end: steps that change nothing
        load_some<BF16>(nx, x + t + off, whole, n, 0.f);
        load_some<BF16>(ni, i + t + off, whole, n, 0.f);
        load_some<BF16>(nd, dout + t + off, whole, n, 0.f);
        if constexpr (GATE)
            load_some<BF16>(nz, z + t + off, whole, n, 0.f);
        if constexpr (RESET)
            nreset = load_resets(reset + t + off, whole, n);
        const int64_t chunk = t / kGatedChunk;
        nstate = p.f.checkpoints[at * chunks + (chunk < chunks ? chunk : chunks - 1)];
    };
    int64_t base = p.f.L > 0 ? start + (stop - 1 - start) / kSpan * kSpan : -1;
    const int64_t mine = wave * (G * kLaneSteps);  // of the wave
    if (base >= 0)
        fetch(base + mine);
    const float rate = row_rate(p.f.c, lam);
    const float rb = row_bias(r_bias), ib = i_bias * kLog2e;
    int turn = 0;
    for (; base >= start; base -= kSpan) {
        const int64_t t = base + mine;
        const Eight<BF16> cx = nx, cr = nr, ci = ni, cz = nz, cd = nd;
        const uint32_t first = nreset;
        const float state = nstate;
        if (base > start)
            fetch(t - kSpan);
        float a[kLaneSteps], u[kLaneSteps], keep_r[kLaneSteps], gate[kLaneSteps], m2[kLaneSteps], rm[kLaneSteps];
        float sum = 0.f, h = 0.f;
        bool dropped = false;
#pragma unroll
        for (int j = 0; j < kLaneSteps; ++j) {
            const float s = sigmoid_log2(cr.get(j), rb);
            keep_r[j] = 1.f - s;
            u[j] = rate * s;
            gate[j] = sigmoid_log2(ci.get(j), ib);
            a[j] = hw_exp2(-u[j]);
            m2[j] = square_of(u[j], a[j]);
            // 1 / m; a step that loses nothing (m = 0) has v = 0, which the floor keeps from 0 / 0
            rm[j] = __builtin_amdgcn_rsqf(fmaxf(m2[j], 1e-37f));
            const float in = gate[j] * cx.get(j);
            sum += u[j];
            h = fmaf(a[j], h, m2[j] * rm[j] * in);
            if (RESET && (first >> j & 1)) {
                h = in;
                dropped = true;
            }
        }
        M m = lane_span<RESET>(sum, dropped, h);
        h = join_before<G, RESET>(m).of(state);
        // h before each step; the output's gradient, through the gate
        float before[kLaneSteps], grad[kLaneSteps], dgate[kLaneSteps];
#pragma unroll
        for (int j = 0; j < kLaneSteps; ++j) {
            before[j] = h;
            const float in = gate[j] * cx.get(j);
            h = fmaf(a[j], h, m2[j] * rm[j] * in);
            if (RESET && (first >> j & 1))
                h = in;
            grad[j] = cd.get(j);
            if constexpr (GATE) {
                const float zj = cz.get(j), sz = sigmoid_log2(zj, 0.f);
                dgate[j] = grad[j] * h * sz * fmaf(zj, 1.f - sz, 1.f);
                grad[j] *= zj * sz;
            }
        }
        float behind = 0.f;
#pragma unroll
        for (int j = kLaneSteps - 1; j >= 0; --j) {
            const float g = grad[j] + behind;
            behind = a[j] * g;
            if (RESET && (first >> j & 1))
                behind = 0.f;
        }
        M back = lane_span<RESET>(sum, dropped, behind);
        const M from = join_behind<G, RESET>(back);
        float enter = carry;
        if constexpr (WAVES > 1) {
            if (lane == 0)
                maps[turn][wave] = float2{back.U, back.S};
            __syncthreads();
#pragma unroll
            for (int w = WAVES - 1; w >= 0; --w) {
                const M other{maps[turn][w].x, maps[turn][w].y};
                carry = other.of(carry);
                if (w - 1 == wave)
                    enter = carry;
            }
            turn ^= 1;
        } else if constexpr (G == 64) {
            carry = read_span(back, 0).of(carry);
        }
        behind = from.of(enter);
        float ox[kLaneSteps], orr[kLaneSteps], oi[kLaneSteps];
#pragma unroll
        for (int j = kLaneSteps - 1; j >= 0; --j) {
            const float g = grad[j] + behind;
            behind = a[j] * g;
            float m1 = m2[j] * rm[j];
            const float in = gate[j] * cx.get(j);
            const float va = u[j] * kLn2 * a[j];  // first: v / m stays small where 1 / m does not
            float q = g * fmaf(va * a[j] * rm[j], in, -va * before[j]);
            if (RESET && (first >> j & 1)) {
                behind = q = 0.f;
                m1 = 1.f;
            }
            ox[j] = g * m1 * gate[j];
            oi[j] = g * m1 * in * (1.f - gate[j]);
            orr[j] = q * keep_r[j];
            sum_q += q;
            sum_r += orr[j];
            sum_i += oi[j];
        }
        const int left = steps_left<G>(L, t), n = lane_share(left, off);
        const bool whole = G == 64 && left == G * kLaneSteps;
        Eight<BF16>::store(dx + t + off, ox, whole, n);
        Eight<BF16>::store(dr + t + off, orr, whole, n);
        Eight<BF16>::store(di + t + off, oi, whole, n);
        if constexpr (GATE)
            Eight<BF16>::store(dz + t + off, dgate, whole, n);
        if (live && t == 0 && lane == 0)
            p.dh0[row] = behind;
    }
    if (p.f.L == 0 && live && lane == 0 && wave == 0)
        p.dh0[row] = carry;
    // a row's sums: over its lanes, then its waves
#pragma unroll
    for (int s = G / 2; s > 0; s >>= 1) {
        sum_q += __shfl_xor(sum_q, s);
        sum_r += __shfl_xor(sum_r, s);
        sum_i += __shfl_xor(sum_i, s);
    }
    if constexpr (WAVES > 1) {
        if (lane == 0) {
            sums[0][wave] = sum_q;
            sums[1][wave] = sum_r;
            sums[2][wave] = sum_i;
        }
        __syncthreads();
        sum_q = sums[0][0];
        sum_r = sums[1][0];
        sum_i = sums[2][0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) {
            sum_q += sums[0][w];
            sum_r += sums[1][w];
            sum_i += sums[2][w];
        }
    }
    if (live && lane == 0 && wave == 0) {
        if (!PARTS && p.f.B == 1) {  // a row's sums are its channel's
            p.dlam[row] = sum_q * lam_slope(lam);
            p.dr_bias[row] = sum_r;
            p.di_bias[row] = sum_i;
        } else {
            const int64_t all = (int64_t)(PARTS ? p.f.parts : 1) * rows;
            float *sum = p.partials + (PARTS ? (int64_t)blockIdx.y * rows : 0) + row;
            sum[0] = sum_q;
            sum[all] = sum_r;
            sum[2 * all] = sum_i;
        }
    }
}

// Sums over the parts and the batch, in their order: a thread a channel and parameter.
__global__ __launch_bounds__(64) void gated_sums_kernel(const GatedScanBwdArgs p)
{
    const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x, count = p.f.parts * p.f.B;
    if (d >= p.f.D)
        return;
    const float *from = p.partials + blockIdx.y * count * p.f.D + d;
    float sum = 0.f;
#pragma unroll 8
    for (int64_t b = 0; b < count; ++b)
        sum += from[b * p.f.D];
    if (blockIdx.y == 0) {
        p.dlam[d] = sum * lam_slope(p.f.lam[d]);
    } else {
        (blockIdx.y == 1 ? p.dr_bias : p.di_bias)[d] = sum;
    }
}

// The maps of a row's parts but the first, for the gradient that runs from the end.
template <bool BF16, bool GATE, bool RESET>
__global__ __launch_bounds__(256) void gated_back_maps_kernel(const GatedScanBwdArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kSpan = 64 * kLaneSteps;
    const int lane = threadIdx.x & 63, part = blockIdx.y + 1;
    const int64_t at = uniform<true>(blockIdx.x * 4 + threadIdx.x / 64);
    if (at >= p.f.B * p.f.D)
        return;
    const uint32_t d = (uint32_t)at % (uint32_t)p.f.D;
    const T *r = (const T *)p.f.r + at * p.f.L, *dout = (const T *)p.dout + at * p.f.L;
    const T *z = GATE ? (const T *)p.f.z + at * p.f.L : nullptr;
    const uint8_t *reset = RESET ? p.f.reset + (int64_t)((uint32_t)at / (uint32_t)p.f.D) * p.f.L : nullptr;
    const float rate = row_rate(p.f.c, p.f.lam[d]);
    const float rb = p.f.r_bias ? row_bias(p.f.r_bias[d]) : 0.f;
    const int64_t start = part * p.f.part_steps, stop = start + p.f.part_steps < p.f.L ? start + p.f.part_steps : p.f.L;
    Span<RESET> all{0.f, 0.f};
    Eight<BF16> nr, nd, nz;
    uint32_t nreset = 0;
    const uint32_t off = lane * kLaneSteps;
    auto fetch = [&](int64_t t) {
        const int left = steps_left<64>(stop, t), n = lane_share(left, off);
        const bool whole = left == kSpan;
        load_some<BF16>(nr, r + t + off, whole, n, -__builtin_inff());
        load_some<BF16>(nd, dout + t + off, whole, n, 0.f);
        if constexpr (GATE)
            load_some<BF16>(nz, z + t + off, whole, n, 0.f);
        if constexpr (RESET)
            nreset = load_resets(reset + t + off, whole, n);
    };
    int64_t base = start + (stop - 1 - start) / kSpan * kSpan;
    fetch(base);
    for (; base >= start; base -= kSpan) {
        const Eight<BF16> cr = nr, cd = nd, cz = nz;
        const uint32_t first = nreset;
        if (base > start)
            fetch(base - kSpan);
        float sum = 0.f, behind = 0.f;
#pragma unroll
        for (int j = kLaneSteps - 1; j >= 0; --j) {
            const float u = rate * sigmoid_log2(cr.get(j), rb);
            float g = cd.get(j);
            if constexpr (GATE)
                g *= cz.get(j) * sigmoid_log2(cz.get(j), 0.f);
            behind = hw_exp2(-u) * (g + behind);
            sum += u;
            if (RESET && (first >> j & 1))
                behind = 0.f;
        }
        Span<RESET> m = lane_span<RESET>(sum, first != 0, behind);
        join_behind<64, RESET>(m);
        Span<RESET> chunk = read_span(m, 0);
        chunk.after(all);
        all = chunk;
    }
    if (lane == 0)
        p.f.maps[at * p.f.parts + part] = float2{all.U, all.S};
}

template <bool BF16, bool GATE, bool RESET> void launch_back_maps(const GatedScanBwdArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.f.B * a.f.D + 3) / 4), a.f.parts - 1), block(256);
    gated_back_maps_kernel<BF16, GATE, RESET><<<grid, block, 0, s>>>(a);
}

template <int G, int WAVES, bool PARTS = false> hipError_t launch(const GatedScanBwdArgs &a, hipStream_t s)
{
    constexpr int kRows = gated_threads(WAVES) / G / WAVES;
    const dim3 grid((unsigned)((a.f.B * a.f.D + kRows - 1) / kRows), PARTS ? a.f.parts : 1), block(gated_threads(WAVES));
    auto with = [&](auto bf16, auto gate, auto reset) {
        if constexpr (PARTS)
            launch_back_maps<bf16, gate, reset>(a, s);
        gated_bwd_kernel<G, WAVES, bf16, gate, reset, PARTS><<<grid, block, 0, s>>>(a);
    };
    auto on_reset = [&](auto bf16, auto gate) {
        if (a.f.reset)
            with(bf16, gate, std::true_type{});
        else
            with(bf16, gate, std::false_type{});
    };
    auto on_gate = [&](auto bf16) {
        if (a.f.z)
            on_reset(bf16, std::true_type{});
        else
            on_reset(bf16, std::false_type{});
    };
    if (a.f.bf16)
        on_gate(std::true_type{});
    else
        on_gate(std::false_type{});
    return hipGetLastError();
}

}  // namespace

// Waves of a row, both sides measured (us, inputs from memory):
//   8 x 5120 x 2048 bf16, gated  one 278, two 334, four 324
//   2 x 1536 x 8192 fp32         one 156, two 150, four 141, eight 155
//   1 x 512 x 32768 bf16         one 102, two 84, four 48, eight 53
//   1 x 1536 x 131072 bf16       one 664, two 634, four 588, eight 544
//   1 x 256 x 131072 bf16, gated one 436, two 231, four 128, eight 119
hipError_t launch_gated_scan_bwd(const GatedScanBwdArgs &a, hipStream_t s)
{
    hipError_t e = hipSuccess;
    const int64_t rows = a.f.B * a.f.D;
    if (rows > 0) {
        switch (gated_group(a.f.L)) {
        case 4: e = launch<4, 1>(a, s); break;
        case 16: e = launch<16, 1>(a, s); break;
        case 32: e = launch<32, 1>(a, s); break;
        default:
            if (a.f.parts > 1) {
                e = launch<64, 1, true>(a, s);
                break;
            }
            switch (gated_waves(rows, a.f.L, a.f.L >= 128 * kGatedChunk ? 8 : 4)) {
            case 1: e = launch<64, 1>(a, s); break;
            case 2: e = launch<64, 2>(a, s); break;
            case 4: e = launch<64, 4>(a, s); break;
            default: e = launch<64, 8>(a, s);
            }
        }
    }
    if (e != hipSuccess || (a.f.B == 1 && a.f.parts == 1))
        return e;
    gated_sums_kernel<<<dim3((unsigned)((a.f.D + 63) / 64), 3), dim3(64), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace mamba
