// Gated linear recurrence, forward: one pass over the inputs (gated_common.h has the
// step).  A lane takes 8 consecutive steps of a row, so its loads and stores are 16
// bytes (bf16) and a wave's are contiguous; G lanes share a row, 64 of them going on
// from chunk to chunk of 512 steps.  Each lane joins its steps to one affine map, the
// wave joins its lanes' maps by DPP, and every lane then runs its steps again from the
// state that enters them.  WAVES waves of a workgroup take consecutive chunks of one
// row, where rows are few; where they are fewer than fill the CUs so, a row is split
// into parts for different workgroups, whose maps a first kernel works out.
//
// What bounds it is memory, with the vector unit close behind (about 40 issue slots an
// element, six of them transcendental at two slots): 8 x 5120 x 2048 bf16 123 us, 5.45
// TB/s, gated 148 with 85 % of the vector unit's slots taken; a large copy moves 5.1 to 5.4.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "gated_common.h"
#include "gated_scan.h"

namespace mamba {
namespace {

// What a lane's eight steps come to, from its inputs as they lie in memory.
template <bool BF16, bool RESET>
__device__ __forceinline__ Span<RESET> lane_steps(const Eight<BF16> &x, const Eight<BF16> &r, const Eight<BF16> &i,
                                                  uint32_t first, float rate, float rb, float ib,
                                                  float (&a)[kLaneSteps], float (&b)[kLaneSteps])
{
    float sum = 0.f, h = 0.f;
    bool dropped = false;
#pragma unroll
    for (int j = 0; j < kLaneSteps; ++j) {
        const float u = rate * sigmoid_log2(r.get(j), rb);
        const float in = sigmoid_log2(i.get(j), ib) * x.get(j);
        a[j] = hw_exp2(-u);
        b[j] = __builtin_amdgcn_sqrtf(square_of(u, a[j])) * in;
        sum += u;
        h = fmaf(a[j], h, b[j]);
        if (RESET && (first >> j & 1)) {
            h = b[j] = in;
            dropped = true;
        }
    }
    return lane_span<RESET>(sum, dropped, h);
}

template <int G, int WAVES, bool BF16, bool GATE, bool RESET, bool PARTS>
__global__ __launch_bounds__(gated_threads(WAVES)) void gated_fwd_kernel(const GatedScanArgs p)
{
    using T = typename Elem<BF16>::T;
    using M = Span<RESET>;
    constexpr int kRows = gated_threads(WAVES) / G / WAVES;  // of a workgroup
    constexpr int kSpan = G * kLaneSteps * WAVES;
    __shared__ float2 maps[2][WAVES];
    const int lane = threadIdx.x & (G - 1), wave = uniform<G == 64>(threadIdx.x / G % WAVES);
    const int rows = (int)(p.B * p.D), row = uniform<G == 64>(blockIdx.x * kRows + threadIdx.x / (G * WAVES));
    const bool live = row < rows;  // the others' lanes run along, with nothing to load or store
    const int64_t from = PARTS ? blockIdx.y * p.part_steps : 0;
    const int64_t stop = PARTS && from + p.part_steps < p.L ? from + p.part_steps : p.L;
    const int64_t at = live ? row : 0, L = live ? stop : 0;
    const uint32_t d = (uint32_t)at % (uint32_t)p.D;  // rows are below 2^24
    const T *x = (const T *)p.x + at * p.L, *r = (const T *)p.r + at * p.L, *i = (const T *)p.i + at * p.L;
    const T *z = GATE ? (const T *)p.z + at * p.L : nullptr;
    T *y = (T *)p.y + at * p.L;
    const uint8_t *reset = RESET ? p.reset + (int64_t)((uint32_t)at / (uint32_t)p.D) * p.L : nullptr;
    const float lam = p.lam[d], r_bias = p.r_bias ? p.r_bias[d] : 0.f, i_bias = p.i_bias ? p.i_bias[d] : 0.f;
    const int64_t chunks = (p.L + kGatedChunk - 1) / kGatedChunk;
    float carry = p.h0 ? p.h0[at] : 0.f;
    if constexpr (PARTS)
        carry = through_parts<RESET>(p.maps + at * p.parts, blockIdx.y, false, p.parts, carry);

    Eight<BF16> nx, nr, ni, nz;
    uint32_t nreset = 0;
    const uint32_t off = lane * kLaneSteps;
    auto fetch = [&](int64_t t) {
        const int left = steps_left<G>(L, t), n = lane_share(left, off);
        const bool whole = G == 64 && left == G * kLaneSteps;
        load_some<BF16>(nr, r + t + off, whole, n, -__builtin_inff());  // past the end: steps that change nothing
        load_some<BF16>(nx, x + t + off, whole, n, 0.f);
        load_some<BF16>(ni, i + t + off, whole, n, 0.f);
        if constexpr (GATE)
            load_some<BF16>(nz, z + t + off, whole, n, 0.f);
        if constexpr (RESET)
            nreset = load_resets(reset + t + off, whole, n);
    };
    int64_t t = from + wave * (G * kLaneSteps);  // of the wave
    fetch(t);
    // worked out while the first loads are on their way
    const float rate = row_rate(p.c, lam);  // of the exponents of 2
    const float rb = row_bias(r_bias), ib = i_bias * kLog2e;
    int turn = 0;
    for (int64_t base = from; base < stop; base += kSpan, t += kSpan) {
        const Eight<BF16> cx = nx, cr = nr, ci = ni, cz = nz;
        const uint32_t first = nreset;
        if (base + kSpan < stop)
            fetch(t + kSpan);
        float a[kLaneSteps], b[kLaneSteps];
        M m = lane_steps<BF16, RESET>(cx, cr, ci, first, rate, rb, ib, a, b);
        const M before = join_before<G, RESET>(m);
        float enter = carry;
        if constexpr (WAVES > 1) {
            if (lane == G - 1)
                maps[turn][wave] = float2{m.U, m.S};
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const M other{maps[turn][w].x, maps[turn][w].y};
                carry = other.of(carry);
                if (w + 1 == wave)
                    enter = carry;
            }
            turn ^= 1;
        } else if constexpr (G == 64) {
            carry = read_span(m, 63).of(carry);
        }
        if (p.checkpoints && lane == 0 && t < L)
            p.checkpoints[at * chunks + t / kGatedChunk] = enter;
        float h = before.of(enter);
        float out[kLaneSteps];
#pragma unroll
        for (int j = 0; j < kLaneSteps; ++j) {
            h = fmaf(a[j], h, b[j]);
            if (RESET && (first >> j & 1))
                h = b[j];
            out[j] = GATE ? h * silu_hw(cz.get(j)) : h;
        }
        if (p.y)
            Eight<BF16>::store(y + t + off, out, G == 64 && steps_left<G>(L, t) == G * kLaneSteps,
                               lane_share(steps_left<G>(L, t), off));
        // the steps past the end have left the state as it was
        if (p.h_last && live && base + kSpan >= p.L && stop == p.L && lane == G - 1 && wave == WAVES - 1)
            p.h_last[row] = h;
    }
    if (p.L == 0 && p.h_last && live && lane == 0 && wave == 0)
        p.h_last[row] = carry;
}

// The maps of a row's parts but the last, a wave each.
template <bool BF16, bool RESET> __global__ __launch_bounds__(256) void gated_maps_kernel(const GatedScanArgs p)
{
    using T = typename Elem<BF16>::T;
    constexpr int kSpan = 64 * kLaneSteps;
    const int lane = threadIdx.x & 63;
    const int64_t at = uniform<true>(blockIdx.x * 4 + threadIdx.x / 64);
    if (at >= p.B * p.D)
        return;
    const uint32_t d = (uint32_t)at % (uint32_t)p.D;
    const T *x = (const T *)p.x + at * p.L, *r = (const T *)p.r + at * p.L, *i = (const T *)p.i + at * p.L;
    const uint8_t *reset = RESET ? p.reset + (int64_t)((uint32_t)at / (uint32_t)p.D) * p.L : nullptr;
    const float rate = row_rate(p.c, p.lam[d]);
    const float rb = p.r_bias ? row_bias(p.r_bias[d]) : 0.f, ib = p.i_bias ? p.i_bias[d] * kLog2e : 0.f;
    const int64_t from = blockIdx.y * p.part_steps;  // whole chunks, and none of them a row's last
    const int64_t stop = from + p.part_steps;
    Span<RESET> all{0.f, 0.f};
    Eight<BF16> nx, nr, ni;
    uint32_t nreset = 0;
    const uint32_t off = lane * kLaneSteps;
    auto fetch = [&](int64_t t) {
        nr.load(r + t + off);
        nx.load(x + t + off);
        ni.load(i + t + off);
        if constexpr (RESET)
            nreset = load_resets(reset + t + off, true, kLaneSteps);
    };
    fetch(from);
    for (int64_t base = from; base < stop; base += kSpan) {
        const Eight<BF16> cx = nx, cr = nr, ci = ni;
        const uint32_t first = nreset;
        if (base + kSpan < stop)
            fetch(base + kSpan);
        float a[kLaneSteps], b[kLaneSteps];
        Span<RESET> m = lane_steps<BF16, RESET>(cx, cr, ci, first, rate, rb, ib, a, b);
        join_before<64, RESET>(m);
        Span<RESET> chunk = read_span(m, 63);
        chunk.after(all);
        all = chunk;
    }
    if (lane == 0)
        p.maps[at * p.parts + blockIdx.y] = float2{all.U, all.S};
}

template <int G, int WAVES, bool PARTS = false> hipError_t launch(const GatedScanArgs &a, hipStream_t s)
{
    constexpr int kRows = gated_threads(WAVES) / G / WAVES;
    const dim3 grid((unsigned)((a.B * a.D + kRows - 1) / kRows), PARTS ? a.parts : 1), block(gated_threads(WAVES));
    auto with = [&](auto bf16, auto gate, auto reset) {
        gated_fwd_kernel<G, WAVES, bf16, gate, reset, PARTS><<<grid, block, 0, s>>>(a);
    };
    auto on_reset = [&](auto bf16, auto gate) {
        if (a.reset)
            with(bf16, gate, std::true_type{});
        else
            with(bf16, gate, std::false_type{});
    };
    auto on_gate = [&](auto bf16) {
        if (a.z)
            on_reset(bf16, std::true_type{});
        else
            on_reset(bf16, std::false_type{});
    };
    if (a.bf16)
        on_gate(std::true_type{});
    else
        on_gate(std::false_type{});
    return hipGetLastError();
}

// ---- one step ----------------------------------------------------------------------------
// A thread takes EACH consecutive channels of one or two sequences (256 x 5120 bf16,
// gated: 8.4 us, 11.8 with one state a thread).  What bounds it is the launch for a few
// sequences, the state's traffic (8 of 18 bytes) and its latency for many.
template <int EACH, bool BF16> struct Few;  // EACH consecutive elements
template <int EACH> struct Few<EACH, true> {
    uint16_t v[EACH];
    __device__ __forceinline__ void load(const uint16_t *p) { __builtin_memcpy(v, p, sizeof(v)); }
    __device__ __forceinline__ float get(int j) const { return bf16_bits_to_f32(v[j]); }
    static __device__ __forceinline__ void store(uint16_t *p, const float (&f)[EACH])
    {
        if constexpr (EACH == 4) {
            const uint32_t w[2] = {cvt2(f[0], f[1]), cvt2(f[2], f[3])};
            __builtin_memcpy(p, w, 8);
        } else {
            Elem<true>::store(p, f[0]);
        }
    }
};
template <int EACH> struct Few<EACH, false> {
    float v[EACH];
    __device__ __forceinline__ void load(const float *p) { __builtin_memcpy(v, p, sizeof(v)); }
    __device__ __forceinline__ float get(int j) const { return v[j]; }
    static __device__ __forceinline__ void store(float *p, const float (&f)[EACH]) { __builtin_memcpy(p, f, sizeof(f)); }
};

template <int EACH, bool BF16, bool GATE>
__global__ __launch_bounds__(256) void gated_step_kernel(const GatedStepArgs p, int64_t parts, int sequences)
{
    using T = typename Elem<BF16>::T;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;  // parts of EACH channels, then sequences
    const int64_t d = n % parts * EACH, b0 = n / parts * sequences;
    if (b0 >= p.B)
        return;
    float rate[EACH], rb[EACH], ib[EACH];
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
        rate[j] = row_rate(p.c, p.lam[d + j]);
        rb[j] = p.r_bias ? row_bias(p.r_bias[d + j]) : 0.f;
        ib[j] = p.i_bias ? p.i_bias[d + j] * kLog2e : 0.f;
    }
    const int64_t end = b0 + sequences < p.B ? b0 + sequences : p.B;
#pragma unroll 2
    for (int64_t b = b0; b < end; ++b) {
        const int64_t at = b * p.D + d;
        Few<EACH, BF16> x, r, i, z;
        Few<EACH, false> h;
        h.load(p.h + at);
        x.load((const T *)p.x + at);
        r.load((const T *)p.r + at);
        i.load((const T *)p.i + at);
        if constexpr (GATE)
            z.load((const T *)p.z + at);
        float state[EACH], y[EACH];
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
            const float u = rate[j] * sigmoid_log2(r.get(j), rb[j]), a = hw_exp2(-u);
            const float in = sigmoid_log2(i.get(j), ib[j]) * x.get(j);
            state[j] = fmaf(a, h.get(j), __builtin_amdgcn_sqrtf(square_of(u, a)) * in);
            y[j] = GATE ? state[j] * silu_hw(z.get(j)) : state[j];
        }
        Few<EACH, false>::store(p.h_out + at, state);
        Few<EACH, BF16>::store((T *)p.y + at, y);
    }
}

template <int EACH> hipError_t launch_step(const GatedStepArgs &a, hipStream_t s)
{
    // two sequences a thread where that leaves every CU eight waves (256 x 5120 bf16,
    // gated: one 9.3 us, two 8.4, four 9.6; 64 x 5120: one 4.8, two 4.6, four 6.1)
    const int64_t parts = a.D / EACH;
    const int sequences = parts * (a.B / 2) >= 256 * 8 * 64 ? 2 : 1;
    const dim3 grid((unsigned)((parts * ((a.B + sequences - 1) / sequences) + 255) / 256)), block(256);
    if (a.bf16 && a.z)
        gated_step_kernel<EACH, true, true><<<grid, block, 0, s>>>(a, parts, sequences);
    else if (a.bf16)
        gated_step_kernel<EACH, true, false><<<grid, block, 0, s>>>(a, parts, sequences);
    else if (a.z)
        gated_step_kernel<EACH, false, true><<<grid, block, 0, s>>>(a, parts, sequences);
    else
        gated_step_kernel<EACH, false, false><<<grid, block, 0, s>>>(a, parts, sequences);
    return hipGetLastError();
}

}  // namespace

// The inputs are then read twice, the second time mostly from the caches.  Both sides
// measured, with waves of one workgroup and in parts (us):
//   1 x 64 x 131072 bf16         55 and 32, backward 85 and 46
//   1 x 32 x 131072 fp32         59 and 29, backward 100 and 43
//   1 x 128 x 131072 bf16, gated 64 and 57, backward 105 and 92 (129 rows, 128 rows)
GatedParts gated_parts(int64_t rows, int64_t L)
{
    const int64_t chunks = (L + kGatedChunk - 1) / kGatedChunk;
    if (rows == 0 || rows > 128 || chunks < 32)
        return {1, L};
    // about 4096 waves in all, four chunks a part or more
    int64_t parts = 4096 / rows < chunks / 4 ? 4096 / rows : chunks / 4;
    parts = parts < 64 ? parts : 64;
    const int64_t each = (chunks + parts - 1) / parts;
    return {(int)((chunks + each - 1) / each), each * kGatedChunk};
}

// Waves of a row, both sides measured (us, inputs from memory):
//   8 x 5120 x 2048 bf16, gated  one 156, two 196, four 182
//   2 x 1536 x 8192 fp32         one 80.3, two 79.9, four 75.8, eight 75.0, 16 83.7
//   1 x 1536 x 131072 bf16       one 401, two 366, four 339, eight 318, 16 365
//   1 x 256 x 131072 bf16, gated one 336, four 89, eight 69, 16 76
//   3 x 771 x 1001 fp32, gated   one 16.4, two 17.0, four 20.0
hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t s)
{
    switch (gated_group(a.L)) {
    case 4: return launch<4, 1>(a, s);
    case 16: return launch<16, 1>(a, s);
    case 32: return launch<32, 1>(a, s);
    }
    const int64_t rows = a.B * a.D;
    if (a.parts > 1) {
        const dim3 grid((unsigned)((rows + 3) / 4), a.parts - 1), block(256);
        if (a.bf16 && a.reset)
            gated_maps_kernel<true, true><<<grid, block, 0, s>>>(a);
        else if (a.bf16)
            gated_maps_kernel<true, false><<<grid, block, 0, s>>>(a);
        else if (a.reset)
            gated_maps_kernel<false, true><<<grid, block, 0, s>>>(a);
        else
            gated_maps_kernel<false, false><<<grid, block, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        return e == hipSuccess ? launch<64, 1, true>(a, s) : e;
    }
    switch (gated_waves(rows, a.L, 8)) {
    case 1: return launch<64, 1>(a, s);
    case 2: return launch<64, 2>(a, s);
    case 4: return launch<64, 4>(a, s);
    default: return launch<64, 8>(a, s);
    }
}

hipError_t launch_gated_step(const GatedStepArgs &a, hipStream_t s)
{
    // four channels a thread where there are enough of them
    return a.D % 4 == 0 && a.B * a.D >= 4 * 256 * 64 ? launch_step<4>(a, s) : launch_step<1>(a, s);
}

}  // namespace mamba
