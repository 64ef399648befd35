// Matrix product of microscaled 4-bit operands:
//   out[m, n] = sum over blocks of 2^(ea[m] + eb[n]) sum_k a[m, k] b[n, k]
// by the matrix cores' scaled instructions, which take a power of two for each row's
// 32 elements beside them; sums in fp32, rounded once to the output type.
//
// Rows are whole groups of 256 elements, a cache line, so a step of both kernels is
// one group: 128 bytes of every row and its 8 scales, all by loads that go from memory
// straight into LDS.
//   tile_kernel  a workgroup's waves share a tile of both operands (256 x 256,
//                128 x 128 or 128 x 64 outputs) and step through the groups together
//   ring_kernel  few output tiles, or few rows on one side: the waves of a workgroup
//                split the groups, each streaming its share through its own LDS ring,
//                and add their sums
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "lds_tiles.h"
#include "mxfp4.h"

namespace mamba {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = kMxGroupBytes;

struct MxParams {
    const uint8_t *a, *b, *a_scale, *b_scale;
    void *out;
    int64_t M, N;
    int groups, row_bytes;
    int64_t a_batch, b_batch;              // rows between batches: 0 = shared
    int64_t a_scale_group, b_scale_group;  // bytes between groups of scales
    int tiles_m, tiles_n;
    int band;                              // tile rows that are walked together
    int64_t tiles;                         // of all batches
};

__device__ __forceinline__ i32x8 wide(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// A wave's loads of 8 * N rows of a tile.  A load takes 8 rows, 8 lanes each; rows past
// the operand's end repeat its last (their products are not stored).
template <int N> struct RowLoads {
    uint32_t off[N];
    __device__ __forceinline__ void set(int first_row, int step_rows, int rows, int row_bytes)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = first_row + i * step_rows + (lane >> 3);
            off[i] = (uint32_t)(row < rows ? row : rows - 1) * (uint32_t)row_bytes + (uint32_t)place(row, lane & 7) * 16;
        }
    }
    __device__ __forceinline__ void issue(uint32_t lds, int step_bytes, const uint8_t *base) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            load_lds(lds + i * step_bytes, base, off[i]);
    }
};

// A wave's loads of the scales of 32 * N rows: 32 rows a load, two lanes a row.
template <int N> struct ScaleLoads {
    uint32_t off[N];
    __device__ __forceinline__ void set(int first_row, int rows)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = first_row + i * 32 + (lane >> 1);
            off[i] = (uint32_t)(row < rows ? row : rows - 1) * kMxScales + (lane & 1) * 4;
        }
    }
    __device__ __forceinline__ void issue(uint32_t lds, const uint8_t *base) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            load_lds4(lds + i * 256, base, off[i]);
    }
};

// ---- large products ------------------------------------------------------------
//
// WM x WN waves of FM x FN blocks of 32 x 32 outputs; STAGES tiles of both operands in
// LDS, the products working on one while the others load.  The workgroup stays for
// several output tiles, and its loads run ahead of the products across the end of a
// tile: the next tile's first stages load while this one's sums are stored.
//
// A step is 4 rounds of 64 elements, two blocks of 32: lanes 0..31 take one, 32..63 the
// other, of a row each.  A round's fragments are read from LDS during the round before,
// a step's scales in the last round before it: 8 bytes a row, of which a lane's round r
// takes byte 2 r + lane / 32.  The one barrier of a step stands before its last round:
// there every wave has read this stage (it may be overwritten) and the next stage has
// arrived.
//
// What bounds it is the card's power, then the rate at which lines reach LDS: 256 x 256
// outputs by 8 waves keep the matrix units busy for 59 % of the cycles at 8192^3 on random
// bytes, at 1.6 GHz (4.2 to 4.4 PFLOP/s); with zeros as data 5.8, which takes 52 bytes a
// ns and CU of the 60 that the caches give all of them.  At 8 x 5120 x 2048 x 2560 (109 to
// 121 us from one card to the next, 45 % busy) power is the smaller part: with zeros as data
// it takes 94 to 99, 4.3 to 4.6 PFLOP/s.  The rest are the tiles' ends, of ten steps each: a
// tile's stores and the loads behind them are counted by one counter, in order, so a step
// after the next waits for the stores.
constexpr int kStaging = 2048;  // of a wave's outputs: 16 rows of 128 bytes
constexpr int scale_loads(int rows, int waves) { return (rows + 32 * waves - 1) / (32 * waves); }
constexpr int stage_bytes(int rows, int waves) { return rows * kStep + scale_loads(rows, waves) * waves * 256; }
constexpr int tile_lds(int WM, int WN, int FM, int FN, int STAGES)
{
    return STAGES * stage_bytes((WM * FM + WN * FN) * 32, WM * WN) + WM * WN * kStaging;
}
// Waves of a SIMD that the LDS leaves room for.
constexpr int tile_waves(int WM, int WN, int FM, int FN, int STAGES)
{
    return 160 * 1024 / tile_lds(WM, WN, FM, FN, STAGES) * WM * WN / 4;
}

template <int WM, int WN, int FM, int FN, int STAGES, bool BF16, bool STREAM>
__global__ __launch_bounds__(64 * WM * WN, tile_waves(WM, WN, FM, FN, STAGES)) void tile_kernel(const MxParams p)
{
    constexpr int TM = WM * FM * 32, TN = WN * FN * 32, NW = WM * WN;
    constexpr int kRowBytes = (TM + TN) * kStep, kStage = stage_bytes(TM + TN, NW);
    constexpr int LA = TM / 8 / NW, LB = TN / 8 / NW;  // loads of a wave and stage
    constexpr int LS = scale_loads(TM + TN, NW), kLoads = LA + LB + LS;
    static_assert(TM % (32 * LS) == 0, "a wave's scales are of one operand");
    constexpr int kWide = BF16 ? 2 : 1;                // blocks of 32 columns in 128 bytes
    constexpr int kStores = FM * FN / kWide * 4;       // of a wave and a whole tile
    static_assert(FN % kWide == 0, "a wave's columns fill whole lines");
    __shared__ __attribute__((aligned(16))) char smem[tile_lds(WM, WN, FM, FN, STAGES)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds;
    const int stride = ((int)gridDim.x - xcd + kXcds - 1) / kXcds;  // workgroups of this XCD
    const Share share = xcd_share(p.tiles, xcd);
    if (slot >= share.count)
        return;
    // Bands of six tile rows, walked along n: 32 neighbouring tiles (an XCD's) then read
    // 6 + 6 operand tiles.  Bands of two (2 + 16) take 4 % more at 8192^3, 8 % more at 5120
    // x 16384 x 2560; one, 16 % more there with 128 x 128 outputs.
    struct Tile {
        int64_t batch, m0, n0;
    };
    auto tile_at = [&](int64_t i) {
        const int64_t id = share.first + i, per = (int64_t)p.tiles_m * p.tiles_n;
        Tile t;
        t.batch = id / per;
        const int rest = (int)(id % per), band = rest / (p.band * p.tiles_n), in = rest % (p.band * p.tiles_n);
        const int left = p.tiles_m - band * p.band, rows = left < p.band ? left : p.band;
        t.m0 = (int64_t)(band * p.band + in % rows) * TM;
        t.n0 = (int64_t)(in / rows) * TN;
        return t;
    };

    // the loads' cursor: STAGES steps ahead of the products
    RowLoads<LA> loads_a;
    RowLoads<LB> loads_b;
    ScaleLoads<LS> loads_s;
    const int scale_row = wave * LS * 32;  // of the tile's rows, a's and then b's
    const bool scales_of_a = scale_row < TM;
    const int64_t scale_group = scales_of_a ? p.a_scale_group : p.b_scale_group;
    const uint8_t *next_a = nullptr, *next_b = nullptr, *next_s = nullptr;
    int64_t load_tile = slot;
    int load_step = 0, ahead = 0;  // ahead: stages issued and not yet waited for
    auto start_tile = [&]() {
        const Tile t = tile_at(load_tile);
        const int64_t ra = t.batch * p.a_batch + t.m0, rb = t.batch * p.b_batch + t.n0;
        const int rows_a = (int)(p.M - t.m0 < TM ? p.M - t.m0 : TM), rows_b = (int)(p.N - t.n0 < TN ? p.N - t.n0 : TN);
        next_a = p.a + ra * p.row_bytes;
        next_b = p.b + rb * p.row_bytes;
        next_s = scales_of_a ? p.a_scale + ra * kMxScales : p.b_scale + rb * kMxScales;
        loads_a.set(wave * 8, NW * 8, rows_a, p.row_bytes);
        loads_b.set(wave * 8, NW * 8, rows_b, p.row_bytes);
        loads_s.set(scales_of_a ? scale_row : scale_row - TM, scales_of_a ? rows_a : rows_b);
    };
    const uint32_t lds = lds_address(smem);
    auto issue = [&](int stage) {
        if (load_tile >= share.count)
            return;
        ++ahead;
        const uint32_t to = lds + stage * kStage;
        loads_a.issue(to + wave * 1024, NW * 1024, next_a);
        loads_b.issue(to + TM * kStep + wave * 1024, NW * 1024, next_b);
        loads_s.issue(to + kRowBytes + scale_row * kMxScales, next_s);
        next_a += kStep;
        next_b += kStep;
        next_s += scale_group;
        if (++load_step == p.groups) {
            load_step = 0;
            load_tile += stride;
            if (load_tile < share.count)
                start_tile();
        }
    };

    // fragments: a lane holds 16 bytes of row lane % 32, half lane / 32
    const int fr = lane & 31, half = lane >> 5;
    auto fragments = [&](i32x4(&fa)[FM], i32x4(&fb)[FN], int stage, int round) {
        const char *s = smem + stage * kStage + fr * kStep + place(fr, round * 2 + half) * 16;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            fa[i] = *(const i32x4 *)(s + (wm * FM + i) * 32 * kStep);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            fb[j] = *(const i32x4 *)(s + (TM + (wn * FN + j) * 32) * kStep);
    };
    u32x2 raw_a[FM], raw_b[FN];  // scales of the step to come
    auto scales = [&](int stage) {
        const char *s = smem + stage * kStage + kRowBytes + fr * kMxScales;
#pragma unroll
        for (int i = 0; i < FM; ++i)
            raw_a[i] = *(const u32x2 *)(s + (wm * FM + i) * 32 * kMxScales);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            raw_b[j] = *(const u32x2 *)(s + (TM + (wn * FN + j) * 32) * kMxScales);
    };

    start_tile();
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        issue(i);
    if (ahead == STAGES)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 1) * kLoads) : "memory");
    else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    --ahead;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    i32x4 fa[2][FM], fb[2][FN];
    fragments(fa[0], fb[0], 0, 0);
    scales(0);
    int stage = 0;
    bool stores_known = false;  // kStores stores were issued behind the last loads
    for (int64_t ti = slot; ti < share.count; ti += stride) {
        const Tile t = tile_at(ti);
        f32x16 acc[FM][FN];
        auto step = [&](auto first) {
            const int next = stage + 1 == STAGES ? 0 : stage + 1;
            int sa[FM][2], sb[FN][2];
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sa[i][h] = (int)(raw_a[i][h] >> (8 * half));
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sb[j][h] = (int)(raw_b[j][h] >> (8 * half));
#pragma unroll
            for (int round = 0; round < 4; ++round) {
                if (round < 3) {
                    fragments(fa[(round + 1) & 1], fb[(round + 1) & 1], stage, round + 1);
                } else {
                    // the products so far stay in front of the barrier
#pragma unroll
                    for (int i = 0; i < FM; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            asm volatile("" : "+v"(acc[i][j]));
                    // The oldest stage in flight has to have arrived: what was
                    // issued behind it may be pending (memory operations count
                    // down in order).  Behind it are the younger stages, or in
                    // a tile's first step of a two-stage kernel the stores of
                    // the tile before.  Where their number is not known,
                    // everything is waited for.
                    if (STAGES > 2 && !first && ahead == STAGES - 1)
                        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * kLoads) : "memory");
                    else if (STAGES == 2 && first && stores_known)
                        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kStores) : "memory");
                    else
                        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    if (ahead > 0)
                        --ahead;
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    fragments(fa[0], fb[0], next, 0);  // after the last step: read, not used
                    scales(next);
                    issue(stage);
                }
                // b's rows on the first side: a lane then holds four
                // consecutive n of one m
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const f32x16 to = first && round == 0 ? f32x16{0} : acc[i][j];
                        const i32x8 vb = wide(fb[round & 1][j]), va = wide(fa[round & 1][i]);
                        const int eb = sb[j][round >> 1], ea = sa[i][round >> 1];
                        if (round & 1)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, to, 4, 4, 2, eb, 2, ea);
                        else
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(vb, va, to, 4, 4, 0, eb, 0, ea);
                    }
                // the reads spread evenly between the products
#pragma unroll
                for (int q = 0; q < FM + FN; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x8, FM * FN / (FM + FN), 0);
                }
            }
            stage = next;
        };
        step(std::true_type{});
        for (int s = 1; s < p.groups; ++s)
            step(std::false_type{});
        // Round and store, 16 rows of 128 bytes at a time through the wave's own piece
        // of LDS, so that a store instruction writes 8 whole lines (in pieces of 64
        // bytes, stores past the caches reach 3.3 TB/s, by whole lines 5.3).  A pass
        // takes half of the lanes' rows: 32 would not fit beside the scales.  In bf16
        // lanes l and l + 32 first exchange, so that each has 8 neighbouring columns.
        using T = typename Elem<BF16>::T;
        constexpr int kPerChunk = BF16 ? 8 : 4;  // elements in 16 bytes
        char *st = smem + STAGES * kStage + wave * kStaging;
        int at = lane;
        asm volatile("" : "+v"(at));  // addresses made anew for each tile: held over the steps, they spill
        const int row16 = at & 15, low = at >> 4 & 1, upper = at >> 5;
        auto finish = [&](auto full) {
#pragma unroll
            for (int j0 = 0; j0 < FN; j0 += kWide) {
                const int64_t n = t.n0 + (wn * FN + j0) * 32 + (at & 7) * kPerChunk;
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    u32x4 w[4];  // chunks of 16 bytes of row fr
                    if constexpr (BF16) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const f32x16 &v = acc[i][j0 + c / 2];
                            const int e = c % 2 * 8;
#pragma unroll
                            for (int d = 0; d < 2; ++d) {
                                const auto x = __builtin_amdgcn_permlane32_swap(
                                    cvt2(v[e + d * 2], v[e + d * 2 + 1]), cvt2(v[e + 4 + d * 2], v[e + 5 + d * 2]), false, false);
                                w[c][d] = x[0];
                                w[c][2 + d] = x[1];
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                w[c][d] = __float_as_uint(acc[i][j0][c * 4 + d]);
                    }
#pragma unroll
                    for (int pass = 0; pass < 2; ++pass) {
                        if (low == pass) {
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                *(u32x4 *)(st + row16 * 128 + place(row16, c * 2 + upper) * 16) = w[c];
                        }
                        asm volatile("" ::: "memory");  // what is read below other lanes have written
                        const int64_t m = t.m0 + (wm * FM + i) * 32 + pass * 16 + (at >> 3);
                        T *o = (T *)p.out + (t.batch * p.M + m) * p.N + n;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int row = r * 8 + (at >> 3);
                            const u32x4 v = *(const u32x4 *)(st + row * 128 + place(row, at & 7) * 16);
                            typedef u32x4 __attribute__((aligned(2))) loose;  // rows start at any element
                            T *to = o + (int64_t)(r * 8) * p.N;
                            if constexpr (full && STREAM) {
                                __builtin_nontemporal_store(v, (loose *)to);
                            } else if constexpr (full) {
                                *(loose *)to = v;
                            } else if (m + r * 8 < p.M) {
                                if (n + kPerChunk <= p.N) {
                                    *(loose *)to = v;
                                } else {
#pragma unroll
                                    for (int q = 0; q < kPerChunk; ++q)
                                        if (n + q < p.N) {
                                            if constexpr (BF16)
                                                to[q] = (uint16_t)(v[q / 2] >> (16 * (q & 1)));
                                            else
                                                to[q] = __uint_as_float(v[q]);
                                        }
                                }
                            }
                        }
                    }
                }
            }
        };
        stores_known = t.m0 + TM <= p.M && t.n0 + TN <= p.N;
        if (stores_known)
            finish(std::true_type{});
        else
            finish(std::false_type{});
    }
}

// ---- few tiles -------------------------------------------------------------------
//
// A workgroup has one tile of FM x FN blocks of 16 x 16 outputs; its NW waves split the
// groups.  No wave waits for another before the sums are added (in the waves' order), so
// the loads of 8 waves run without a common pause.
template <int FM, int FN, int STAGES, bool BF16> __global__ __launch_bounds__(512) void ring_kernel(const MxParams p)
{
    constexpr int NW = 8, TM = FM * 16, TN = FN * 16, SA = (TM + 31) / 32, SB = (TN + 31) / 32;
    constexpr int kRowBytes = (TM + TN) * kStep, kStage = kRowBytes + (SA + SB) * 256;
    constexpr int kLoads = 2 * (FM + FN) + SA + SB;
    __shared__ __attribute__((aligned(16))) char smem[NW * STAGES * kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Share share = xcd_share(p.tiles, blockIdx.x % kXcds);
    const int64_t id = share.first + blockIdx.x / kXcds, per = (int64_t)p.tiles_m * p.tiles_n;
    const int64_t batch = id / per;
    const int rest = (int)(id % per);
    const int64_t m0 = (int64_t)(rest % p.tiles_m) * TM, n0 = (int64_t)(rest / p.tiles_m) * TN;
    const int64_t ra = batch * p.a_batch + m0, rb = batch * p.b_batch + n0;
    const uint8_t *a = p.a + ra * p.row_bytes, *b = p.b + rb * p.row_bytes;
    const uint8_t *a_scale = p.a_scale + ra * kMxScales, *b_scale = p.b_scale + rb * kMxScales;
    const int rows_a = (int)(p.M - m0 < TM ? p.M - m0 : TM), rows_b = (int)(p.N - n0 < TN ? p.N - n0 : TN);
    RowLoads<2 * FM> loads_a;
    RowLoads<2 * FN> loads_b;
    ScaleLoads<SA> scales_a;
    ScaleLoads<SB> scales_b;
    loads_a.set(0, 8, rows_a, p.row_bytes);
    loads_b.set(0, 8, rows_b, p.row_bytes);
    scales_a.set(0, rows_a);
    scales_b.set(0, rows_b);

    const int each = (p.groups + NW - 1) / NW, from = wave * each;
    const int to = from + each < p.groups ? from + each : p.groups;
    char *mine = smem + wave * STAGES * kStage;
    const uint32_t lds = lds_address(mine);
    auto issue = [&](int step, int stage) {
        const uint32_t l = lds + stage * kStage;
        loads_a.issue(l, 1024, a + (int64_t)step * kStep);
        loads_b.issue(l + TM * kStep, 1024, b + (int64_t)step * kStep);
        scales_a.issue(l + kRowBytes, a_scale + step * p.a_scale_group);
        scales_b.issue(l + kRowBytes + SA * 256, b_scale + step * p.b_scale_group);
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        if (from + i < to)
            issue(from + i, i);
    // fragments: a lane holds 16 bytes of row lane % 16, quarter lane / 16
    const int fr = lane & 15, quarter = lane >> 4;
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int stage = 0;
    for (int s = from; s < to; ++s) {
        if (s + STAGES <= to)  // arrived when only the younger stages' loads are pending
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads * (STAGES - 1)) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        i32x4 fa[2][FM], fb[2][FN];
        u32x2 sa[FM], sb[FN];
        const char *at = mine + stage * kStage;
#pragma unroll
        for (int round = 0; round < 2; ++round) {
            const char *f = at + fr * kStep + place(fr, round * 4 + quarter) * 16;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[round][i] = *(const i32x4 *)(f + i * 16 * kStep);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[round][j] = *(const i32x4 *)(f + (TM + j * 16) * kStep);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i)
            sa[i] = *(const u32x2 *)(at + kRowBytes + (i * 16 + fr) * kMxScales);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            sb[j] = *(const u32x2 *)(at + kRowBytes + SA * 256 + (j * 16 + fr) * kMxScales);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the stage may be overwritten
        if (s + STAGES < to)
            issue(s + STAGES, stage);
#pragma unroll
        for (int round = 0; round < 2; ++round)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        wide(fb[round][j]), wide(fa[round][i]), acc[i][j], 4, 4, 0, (int)(sb[j][round] >> (8 * quarter)), 0,
                        (int)(sa[i][round] >> (8 * quarter)));
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // Each wave's sums go where its steps lay: blocks of 16 x 16, of which a lane
    // holds four consecutive n of one m.  `spread` lets 16 lanes write one quarter
    // of a block, and 16 lanes read consecutive n, from different banks.
    constexpr int kWaveBytes = STAGES * kStage;
    static_assert(TM * TN * 4 <= kWaveBytes, "a wave's sums take its ring's place");
    auto spread = [](int i, int j, int q, int r) {
        const int x = FN <= 2 ? (j * 4 + q) * (4 / FN) : j * 4 + q;
        return ((i * FN + j) * 64 + q * 16 + (r ^ x)) * 16;
    };
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            *(f32x4 *)(mine + spread(i, j, quarter, fr)) = acc[i][j];
    __syncthreads();
    // four consecutive n of one m a thread
    using T = typename Elem<BF16>::T;
    T *out = (T *)p.out + (batch * p.M + m0) * p.N + n0;
    for (int i = threadIdx.x; i < TM * TN / 4; i += 64 * NW) {
        const int m = i / (TN / 4), n = i % (TN / 4) * 4;
        if (m >= rows_a || n >= rows_b)
            continue;
        const char *part = smem + spread(m / 16, n / 16, n % 16 / 4, m % 16);
        f32x4 sum = *(const f32x4 *)part;
#pragma unroll
        for (int w = 1; w < NW; ++w)
            sum += *(const f32x4 *)(part + w * kWaveBytes);
        T *o = out + (int64_t)m * p.N + n;
        if (n + 4 <= rows_b) {
            if constexpr (BF16) {
                const u32x2 w = {cvt2(sum[0], sum[1]), cvt2(sum[2], sum[3])};
                __builtin_memcpy(o, &w, 8);
            } else {
                __builtin_memcpy(o, &sum, 16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < rows_b)
                    Elem<BF16>::store(o + e, sum[e]);
        }
    }
}

// Products of no channels.
template <bool BF16> __global__ __launch_bounds__(256) void zero_kernel(void *out, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        Elem<BF16>::store((typename Elem<BF16>::T *)out + i, 0.f);
}

// ---- choice --------------------------------------------------------------------------
//
// Which tile: the one whose time, by this model, is least, in us:
//   max(rounds * steps * alone, tiles / slots * steps * busy) + rounds * each + once
// rounds: output tiles a workgroup slot takes after one another; alone: a step of one
// group on an otherwise free card; busy: with every slot taken, where power and the
// shared caches hold the rate; each: a tile's end.  The constants are fitted to 1000
// shapes drawn from 1 x 16 to 65536 x 8192 with 64 to 8192 of the inner axis, each timed
// in every form, when tiles were walked in bands of two rows.  Bands of six made the large
// products 4 to 8 % faster; of 1000 other shapes timed with them the form chosen takes 1.7 %
// more than the fastest on average, 4.6 % at the ninetieth percentile, and 35 % at the worst
// (8121 x 25236 x 107: 145 us, 108 by 128 x 128 tiles of four stages).  Both sides of some
// of the choices, in us:
//   8 x 5120 x 2048 x 2560   256 x 256 tiles 116, 128 x 128 146
//   16384 x 1536 x 768       128 x 128 tiles of two stages 18.7, 256 x 256 20.5, 128 x 64 40.5
//   256 x 5120 x 2560        128 x 128 tiles of two stages 9.3, of four 9.6, rings of 48 x 64 9.9
//   512 x 1536 x 768         rings of 64 x 48 4.5, of 48 x 64 6.4, 128 x 128 tiles 5.4
//   256 x 2560 x 5120        rings of 64 x 48 7.1, of 64 x 64 7.9, 128 x 128 tiles 13.9
//   64 x 2560 x 5120         rings of 32 x 32 4.7, of 32 x 64 5.6, of 16 x 16 6.3
//   1 x 5120 x 2560          rings of 16 x 32 3.7, of 32 x 32 4.3, of 64 x 64 5.7, 128 x 128 tiles 8.9
enum Form { kTile256, kTile128, kTile128Deep, kTile64, kRing44, kRing34, kRing43, kRing24, kRing42, kRing22, kRing12, kRing21, kRing11, kForms };
struct FormCost {
    int tm, tn, slots;
    double alone, busy, each, once;
};
// A ring's loads bound it, alone or not.
constexpr FormCost ring_cost(int tm, int tn)
{
    return FormCost{tm, tn, kCus, .0014 * (tm + tn), .0014 * (tm + tn), 1.32 + .000135 * tm * tn, 2.17};
}
constexpr FormCost kCosts[kForms] = {{256, 256, kCus, 1.51, 1.54, 5.93, 2.63},
                                     {128, 128, 2 * kCus, 0.63, 1.16, 2.62, 1.92},
                                     {128, 128, kCus, 0.45, 0.64, 2.07, 2.35},
                                     {128, 64, kCus, 0.49, 0.50, 1.49, 2.34},
                                     ring_cost(64, 64), ring_cost(48, 64), ring_cost(64, 48), ring_cost(32, 64), ring_cost(64, 32),
                                     ring_cost(32, 32), ring_cost(16, 32), ring_cost(32, 16), ring_cost(16, 16)};
constexpr int64_t kMostRingTiles = 1 << 16;  // of 512 threads

int64_t tiles_of(const FormCost &f, int64_t batch, int64_t M, int64_t N)
{
    return batch * ((M + f.tm - 1) / f.tm) * ((N + f.tn - 1) / f.tn);
}

Form choose(int64_t batch, int64_t M, int64_t N, int64_t groups)
{
    Form best = kTile128;
    double least = -1.;
    for (int f = kTile256; f < kForms; ++f) {
        const FormCost &c = kCosts[f];
        const int64_t tiles = tiles_of(c, batch, M, N);
        if (f >= kRing44 && tiles > kMostRingTiles)
            continue;
        const double rounds = (double)((tiles + c.slots - 1) / c.slots), steps = (double)groups;
        const double alone = rounds * c.alone, busy = (double)tiles / c.slots * c.busy;
        const double cost = steps * (alone > busy ? alone : busy) + rounds * c.each + c.once;
        if (least < 0. || cost < least) {
            best = (Form)f;
            least = cost;
        }
    }
    return best;
}

template <int WM, int WN, int FM, int FN, int STAGES> hipError_t tile(const MxParams &p, int slots, bool bf16, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles < slots ? p.tiles : slots)), block(64 * WM * WN);
    // Rows that start at 64-byte boundaries are stored past the caches in whole
    // pieces of memory traffic; others leave pieces that a cache has to join.
    const bool stream = (p.N * (bf16 ? 2 : 4)) % 64 == 0 && (uintptr_t)p.out % 64 == 0;
    if (bf16 && stream)
        tile_kernel<WM, WN, FM, FN, STAGES, true, true><<<grid, block, 0, s>>>(p);
    else if (bf16)
        tile_kernel<WM, WN, FM, FN, STAGES, true, false><<<grid, block, 0, s>>>(p);
    else if (stream)
        tile_kernel<WM, WN, FM, FN, STAGES, false, true><<<grid, block, 0, s>>>(p);
    else
        tile_kernel<WM, WN, FM, FN, STAGES, false, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <int FM, int FN, int STAGES> hipError_t ring(const MxParams &p, bool bf16, hipStream_t s)
{
    const dim3 grid((unsigned)p.tiles), block(512);
    if (bf16)
        ring_kernel<FM, FN, STAGES, true><<<grid, block, 0, s>>>(p);
    else
        ring_kernel<FM, FN, STAGES, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

MxMatmulForm mxfp4_matmul_form(const MxMatmulArgs &a)
{
    // one right operand for every batch: the batches' rows follow one another
    const bool joined = a.b_shared && !a.a_shared;
    MxMatmulForm r{};
    r.batch = joined ? 1 : a.batch;
    r.M = joined ? a.batch * a.M : a.M;
    r.form = choose(r.batch, r.M, a.N, a.groups);
    const FormCost &c = kCosts[r.form];
    r.slots = c.slots;
    r.tile_m = c.tm;
    r.tile_n = c.tn;
    r.tiles = tiles_of(c, r.batch, r.M, a.N);
    return r;
}

hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, hipStream_t s)
{
    if (a.groups == 0) {
        const int64_t n = a.batch * a.M * a.N, blocks = (n + 255) / 256;
        const dim3 grid((unsigned)(blocks < 8 * kCus ? blocks : 8 * kCus)), block(256);
        if (a.bf16)
            zero_kernel<true><<<grid, block, 0, s>>>(a.out, n);
        else
            zero_kernel<false><<<grid, block, 0, s>>>(a.out, n);
        return hipGetLastError();
    }
    const MxMatmulForm f = mxfp4_matmul_form(a);
    MxParams p{};
    p.a = a.a;
    p.b = a.b;
    p.a_scale = a.a_scale;
    p.b_scale = a.b_scale;
    p.out = a.out;
    p.M = f.M;
    p.N = a.N;
    p.groups = (int)a.groups;
    p.row_bytes = (int)a.groups * kMxGroupBytes;
    p.a_batch = a.a_shared ? 0 : f.M;
    p.b_batch = a.b_shared ? 0 : a.N;
    p.a_scale_group = (a.a_shared ? a.M : a.batch * a.M) * kMxScales;
    p.b_scale_group = (a.b_shared ? a.N : a.batch * a.N) * kMxScales;
    p.tiles_m = (int)((f.M + f.tile_m - 1) / f.tile_m);
    p.tiles_n = (int)((a.N + f.tile_n - 1) / f.tile_n);
    p.band = p.tiles_m < 6 ? p.tiles_m : 6;
    p.tiles = f.tiles;
    switch (f.form) {
    case kTile256: return tile<2, 4, 4, 2, 2>(p, f.slots, a.bf16, s);
    case kTile128: return tile<2, 2, 2, 2, 2>(p, f.slots, a.bf16, s);
    case kTile128Deep: return tile<4, 2, 1, 2, 4>(p, f.slots, a.bf16, s);
    case kTile64: return tile<4, 1, 1, 2, 3>(p, f.slots, a.bf16, s);
    case kRing44: return ring<4, 4, 1>(p, a.bf16, s);
    case kRing43: return ring<4, 3, 1>(p, a.bf16, s);
    case kRing34: return ring<3, 4, 1>(p, a.bf16, s);
    case kRing42: return ring<4, 2, 1>(p, a.bf16, s);
    case kRing24: return ring<2, 4, 1>(p, a.bf16, s);
    case kRing22: return ring<2, 2, 2>(p, a.bf16, s);
    case kRing12: return ring<1, 2, 2>(p, a.bf16, s);
    case kRing21: return ring<2, 1, 2>(p, a.bf16, s);
    default: return ring<1, 1, 2>(p, a.bf16, s);
    }
}

}  // namespace mamba
