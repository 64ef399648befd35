// Matrix product of 8-bit integers with a scale for each row of both operands:
//   out[m, n] = a_scale[m] b_scale[n] sum_k a[m, k] b[n, k]
// The sum is exact (32-bit integers); it is converted to fp32, scaled, and
// rounded once to the output type.
//
// Two kernels, both with the operand rows in LDS in tiles of 128 bytes (one
// cache line) of the inner axis, both fed by loads that go from memory straight
// into LDS (DIRECT, global_load_lds_dwordx4: no registers, so as many are in
// flight as LDS holds), or, where rows do not start at 16-byte boundaries, which
// those loads need, by way of registers:
//   tile_kernel  a workgroup's waves share a tile of both operands (256 x 256,
//                128 x 128 or 128 x 64 outputs) and step through the inner axis together
//   ring_kernel  few output tiles, or few rows on one side: the waves of a
//                workgroup split the inner axis, each streaming its share
//                through its own LDS ring, and add their integer sums
#include <hip/hip_runtime.h>

#include <type_traits>

#include "device_common.h"
#include "lds_tiles.h"
#include "quant.h"

namespace mamba {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;     // bytes of the inner axis a step takes: a cache line of every row

struct MatmulParams {
    const int8_t *a, *b;
    const float *a_scale, *b_scale;
    void *out;
    int64_t M, N;
    int K, steps;              // steps of kStep bytes, at least 1 (K = 0: all zeros)
    int64_t a_batch, b_batch;  // rows between batches: 0 = shared
    int tiles_m, tiles_n;
    int64_t tiles;             // of all batches
};

// Past the inner axis' end a lane loads these instead.
__device__ const u32x4 kZeros = {0, 0, 0, 0};

// The 16 bytes that end a row of K bytes (K >= 16) moved down so that its last
// `rem` come first, zeros behind them.
__device__ __forceinline__ u32x4 row_end(u32x4 v, int rem)
{
    const int shift = 16 - rem, words = shift >> 2;
    uint32_t w[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = i; j < 4; ++j)
            w[i] = j - i == words ? v[j] : w[i];
    }
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], shift & 3);
    return r;
}

// A wave's loads of 8 * N rows of a tile.  A load takes 8 rows, 8 lanes each;
// rows past the operand's end repeat its last (their products are not stored).
// Past the inner axis' end LDS gets zeros.
template <int N, bool DIRECT> struct RowLoads {
    uint32_t off[N];
    u32x4 held[DIRECT ? 1 : N];
    __device__ __forceinline__ void set(int first_row, int step_rows, int rows, int K)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = first_row + i * step_rows + (lane >> 3);
            off[i] = (uint32_t)((row < rows ? row : rows - 1) * K + place(row, lane & 7) * 16);
        }
    }
    // DIRECT: a whole step into LDS.
    __device__ __forceinline__ void whole(uint32_t lds, int step_bytes, const int8_t *base) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            load_lds(lds + i * step_bytes, base, off[i]);
    }
    // DIRECT: the last step of an inner axis that is no multiple of kStep, of
    // which `left` bytes are left.
    __device__ __forceinline__ void partial(uint32_t lds, int step_bytes, const int8_t *base, int first_row,
                                            int step_rows, int left) const
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int row = first_row + i * step_rows + (lane >> 3);
            const int8_t *p = place(row, lane & 7) * 16 < left ? base + off[i] : (const int8_t *)&kZeros;
            load_lds(lds + i * step_bytes, p);
        }
    }
    // By way of registers: fetch a step of which `left` bytes are left, then
    // put it into LDS.
    __device__ __forceinline__ void fetch(const int8_t *base, int first_row, int step_rows, int left, int K)
    {
        const int lane = threadIdx.x & 63;
        if (left >= kStep) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                __builtin_memcpy(&held[i], base + off[i], 16);
        } else if (K >= 16) {
            // a chunk that passes the row's end is read so as to end with it
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = left - place(first_row + i * step_rows + (lane >> 3), lane & 7) * 16;
                u32x4 v;
                __builtin_memcpy(&v, base + (int64_t)off[i] + (r < 16 ? r - 16 : 0), 16);
                const u32x4 end = row_end(v, left & 15);
                held[i] = r >= 16 ? v : (r > 0 ? end : u32x4{0, 0, 0, 0});
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = left - place(first_row + i * step_rows + (lane >> 3), lane & 7) * 16;
                uint64_t lo = 0, hi = 0;
#pragma unroll 1
                for (int j = 0; j < r; ++j) {
                    const uint64_t byte = (uint64_t)(uint8_t)base[off[i] + j] << (8 * (j & 7));
                    lo |= j < 8 ? byte : 0;
                    hi |= j < 8 ? 0 : byte;
                }
                held[i] = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
            }
        }
    }
    __device__ __forceinline__ void put(char *to, int step_bytes) const
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < N; ++i)
            *(u32x4 *)(to + i * step_bytes + lane * 16) = held[i];
    }
};

// ---- large products ------------------------------------------------------------
//
// WM x WN waves of FM x FN blocks of 32 x 32 outputs; STAGES tiles of both
// operands in LDS, the products working on one while the others load.  The
// workgroup stays for several output tiles, and its loads run ahead of the
// products across the end of a tile: the next tile's first stages load while
// this one's sums are scaled and stored.
//
// A step is 4 rounds of 32 bytes; a round's fragments are read from LDS during
// the round before.  The one barrier of a step stands before its last round:
// there every wave has read this stage (it may be overwritten) and the next
// stage has arrived.
//
// What bounds it is the card's power: 256 x 256 outputs by 8 waves keep the
// matrix units busy for 68 % of the cycles at 8192^3 on random data, at clocks
// that go down to 1.85 GHz (2.28 to 2.45 POP/s from card to card and run to run,
// where the library's 8-bit product reaches 2.14).  With zeros as data the clock
// stays at 2.4 GHz; without any loads, on random data, the products alone reach
// 2.75.  LDS is read a quarter of the time, nearly without bank conflicts.  Of a
// tile's end most is arithmetic (3.5 instructions an output) and the stores' way
// to memory: whole lines past the caches, issued without branches, and not waited
// for by the next tile's first step (8 x 5120 x 2048 x 2560, on one card: 178 us,
// by way of the caches 204; before also guarded, waited for, and with the scales
// loaded there 212; from card to card and with a trace running, 178 to 212).
constexpr int kStaging = 4096;  // of a wave's outputs: 32 rows of 128 bytes
constexpr int tile_lds(int WM, int WN, int FM, int FN, int STAGES)
{
    return STAGES * (WM * FM + WN * FN) * 32 * kStep + WM * WN * kStaging;
}
// Waves of a SIMD that the LDS leaves room for: 2, or 1 for tiles of 128 x 64
// (88 KB, so one workgroup of four waves a CU).
constexpr int tile_waves(int WM, int WN, int FM, int FN, int STAGES)
{
    return 160 * 1024 / tile_lds(WM, WN, FM, FN, STAGES) * WM * WN / 4;
}

template <int WM, int WN, int FM, int FN, int STAGES, bool DIRECT, bool BF16, bool STREAM>
__global__ __launch_bounds__(64 * WM * WN, tile_waves(WM, WN, FM, FN, STAGES)) void tile_kernel(const MatmulParams p)
{
    constexpr int TM = WM * FM * 32, TN = WN * FN * 32, NW = WM * WN;
    constexpr int kStage = (TM + TN) * kStep;
    constexpr int LA = TM / 8 / NW, LB = TN / 8 / NW;  // loads of a wave and stage
    constexpr int SA = (FM + 1) / 2, SB = (FN + 1) / 2;  // registers of a wave's scales
    constexpr int kWide = BF16 ? 2 : 1;                // blocks of 32 columns in 128 bytes
    constexpr int kPerChunk = BF16 ? 8 : 4;            // elements in 16 bytes
    constexpr int kStores = FM * 4 * (FN / kWide);     // of a wave and a whole tile
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
    // Bands of two tile rows, walked along n: 32 neighbouring tiles (an XCD's)
    // then read 2 + 16 operand tiles.  Bands of 1..8 rows at four shapes: 2 is
    // never more than 1 % behind the best; 1 loses 15 % at 8192^3.
    constexpr int kBand = 2;
    struct Tile {
        int64_t batch, m0, n0;
    };
    auto tile_at = [&](int64_t i) {
        const int64_t id = share.first + i, per = (int64_t)p.tiles_m * p.tiles_n;
        Tile t;
        t.batch = id / per;
        const int rest = (int)(id % per), band = rest / (kBand * p.tiles_n), in = rest % (kBand * p.tiles_n);
        const int left = p.tiles_m - band * kBand, rows = left < kBand ? left : kBand;
        t.m0 = (int64_t)(band * kBand + in % rows) * TM;
        t.n0 = (int64_t)(in / rows) * TN;
        return t;
    };

    // the loads' cursor: STAGES steps ahead of the products, one more by way of registers
    RowLoads<LA, DIRECT> loads_a;
    RowLoads<LB, DIRECT> loads_b;
    const int8_t *next_a = nullptr, *next_b = nullptr;
    int64_t load_tile = slot;
    int load_step = 0, ahead = 0;  // ahead: stages issued and not yet waited for
    auto start_tile = [&]() {
        const Tile t = tile_at(load_tile);
        next_a = p.a + (t.batch * p.a_batch + t.m0) * p.K;
        next_b = p.b + (t.batch * p.b_batch + t.n0) * p.K;
        loads_a.set(wave * 8, NW * 8, (int)(p.M - t.m0 < TM ? p.M - t.m0 : TM), p.K);
        loads_b.set(wave * 8, NW * 8, (int)(p.N - t.n0 < TN ? p.N - t.n0 : TN), p.K);
    };
    auto advance = [&]() {
        next_a += kStep;
        next_b += kStep;
        if (++load_step == p.steps) {
            load_step = 0;
            load_tile += stride;
            if (load_tile < share.count)
                start_tile();
        }
    };
    bool holds = false;  // a step waits in registers
    auto fetch = [&]() {
        holds = load_tile < share.count;
        if (!holds)
            return;
        const int left = p.K - load_step * kStep;
        loads_a.fetch(next_a, wave * 8, NW * 8, left, p.K);
        loads_b.fetch(next_b, wave * 8, NW * 8, left, p.K);
        advance();
    };
    const uint32_t lds = lds_address(smem) + wave * 1024;
    auto issue = [&](int stage) {
        if constexpr (DIRECT) {
            if (load_tile >= share.count)
                return;
            ++ahead;
            const uint32_t to = lds + stage * kStage;
            const int left = p.K - load_step * kStep;
            if (left >= kStep) {
                loads_a.whole(to, NW * 1024, next_a);
                loads_b.whole(to + TM * kStep, NW * 1024, next_b);
            } else {
                loads_a.partial(to, NW * 1024, next_a, wave * 8, NW * 8, left);
                loads_b.partial(to + TM * kStep, NW * 1024, next_b, wave * 8, NW * 8, left);
            }
            advance();
        } else if (holds) {
            char *to = smem + stage * kStage + wave * 1024;
            loads_a.put(to, NW * 1024);
            loads_b.put(to + TM * kStep, NW * 1024);
            fetch();
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

    start_tile();
    if constexpr (!DIRECT)
        fetch();
#pragma unroll
    for (int i = 0; i < STAGES; ++i)
        issue(i);
    if constexpr (DIRECT) {
        if (ahead == STAGES)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 1) * (LA + LB)) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        --ahead;
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    i32x4 fa[2][FM], fb[2][FN];
    fragments(fa[0], fb[0], 0, 0);
    int stage = 0;
    bool stores_known = false;  // kStores stores were issued behind the last loads
    for (int64_t ti = slot; ti < share.count; ti += stride) {
        const Tile t = tile_at(ti);
        // this wave's scales, a row or column a lane; they wait here for the end of the tile
        const float *a_scale = p.a_scale + t.batch * p.a_batch, *b_scale = p.b_scale + t.batch * p.b_batch;
        float sa[SA], sb[SB];
#pragma unroll
        for (int i = 0; i < SA; ++i) {
            const int64_t m = t.m0 + wm * FM * 32 + i * 64 + lane;
            sa[i] = a_scale[m < p.M ? m : p.M - 1];
        }
#pragma unroll
        for (int i = 0; i < SB; ++i) {
            const int64_t n = t.n0 + wn * FN * 32 + i * 64 + lane;
            sb[i] = b_scale[n < p.N ? n : p.N - 1];
        }
        i32x16 acc[FM][FN];
        auto step = [&](int s, auto first) {
            const int next = stage + 1 == STAGES ? 0 : stage + 1;
#pragma unroll
            for (int round = 0; round < 4; ++round) {
                if (round < 3) {
                    fragments(fa[(round + 1) & 1], fb[(round + 1) & 1], stage, round + 1);
                } else {
                    if (DIRECT && s == p.steps - 1) {  // the scales have arrived long since: the compiler's wait for them
#pragma unroll
                        for (int i = 0; i < SA; ++i)
                            asm volatile("" : "+v"(sa[i]));
#pragma unroll
                        for (int i = 0; i < SB; ++i)
                            asm volatile("" : "+v"(sb[i]));
                    }
                    // The oldest stage in flight has to have arrived: what was
                    // issued behind it may be pending (memory operations count
                    // down in order).  Behind it are the younger stages, or in
                    // a tile's first step of a two-stage kernel the stores of
                    // the tile before.  Where their number is not known,
                    // everything is waited for.
                    if constexpr (DIRECT) {
                        if (STAGES > 2 && !first && ahead == STAGES - 1)
                            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((STAGES - 2) * (LA + LB)) : "memory");
                        else if (STAGES == 2 && first && stores_known)
                            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kStores) : "memory");
                        else
                            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                        if (ahead > 0)
                            --ahead;
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    fragments(fa[0], fb[0], next, 0);  // after the last step: read, not used
                    issue(stage);
                }
                // b's rows on the first side: a lane then holds four
                // consecutive n of one m
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const i32x16 to = first && round == 0 ? i32x16{0} : acc[i][j];
                        acc[i][j] =
                            __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[round & 1][j], fa[round & 1][i], to, 0, 0, 0);
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
        step(0, std::true_type{});
        for (int s = 1; s < p.steps; ++s)
            step(s, std::false_type{});
        // Scale and store, 32 rows of 128 bytes at a time through the wave's
        // own piece of LDS, so that a store instruction writes 8 whole lines
        // (straight from the registers it would touch 32 rows, 16 bytes each:
        // 40 us more at 8 x 5120 x 2048 x 2560).
        using T = typename Elem<BF16>::T;
        char *st = smem + STAGES * kStage + wave * kStaging;
#pragma unroll
        for (int i = 0; i < SA; ++i)
            ((float *)st)[i * 64 + lane] = sa[i];
#pragma unroll
        for (int i = 0; i < SB; ++i)
            ((float *)st)[(SA + i) * 64 + lane] = sb[i];
        float row_scale[FM];
        f32x4 col_scale[FN][4];
#pragma unroll
        for (int i = 0; i < FM; ++i)
            row_scale[i] = ((const float *)st)[i * 32 + fr];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                col_scale[j][e] = *(const f32x4 *)(st + (SA * 64 + j * 32 + e * 8 + half * 4) * 4);
        auto finish = [&](auto full) {
#pragma unroll
            for (int j0 = 0; j0 < FN; j0 += kWide) {
                const int64_t n = t.n0 + (wn * FN + j0) * 32 + (lane & 7) * kPerChunk;
                const int64_t m = t.m0 + wm * FM * 32 + (lane >> 3);
                T *o = (T *)p.out + (t.batch * p.M + m) * p.N + n;
#pragma unroll
                for (int i = 0; i < FM; ++i) {
#pragma unroll
                    for (int j = 0; j < kWide; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                v[q] = (float)acc[i][j0 + j][e * 4 + q] * row_scale[i] * col_scale[j0 + j][e][q];
                            if constexpr (BF16) {
                                const u32x2 w = {cvt2(v[0], v[1]), cvt2(v[2], v[3])};
                                *(u32x2 *)(st + fr * 128 + place(fr, j * 4 + e) * 16 + half * 8) = w;
                            } else {
                                const u32x4 w = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                                 __float_as_uint(v[3])};
                                *(u32x4 *)(st + fr * 128 + place(fr, e * 2 + half) * 16) = w;
                            }
                        }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = r * 8 + (lane >> 3);
                        const u32x4 v = *(const u32x4 *)(st + row * 128 + place(row, lane & 7) * 16);
                        typedef u32x4 __attribute__((aligned(2))) loose;  // rows start at any element
                        T *to = o + (int64_t)(i * 32 + r * 8) * p.N;
                        if constexpr (full && STREAM) {
                            __builtin_nontemporal_store(v, (loose *)to);
                        } else if constexpr (full) {
                            *(loose *)to = v;
                        } else if (m + i * 32 + r * 8 < p.M) {
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
// A workgroup has one tile of FM x FN blocks of 16 x 16 outputs; its NW waves
// split the inner axis.  No wave waits for another before the sums are added
// (integers: in any order), so the loads of 8 waves, 128 KB a workgroup, run
// without a common pause.  What bounds it is the rate at which one CU takes
// lines into LDS (a single workgroup on an idle card: 97 bytes a ns, all of
// them together about 60) and, for one token, the launch.
template <int FM, int FN, int STAGES, bool DIRECT, bool BF16>
__global__ __launch_bounds__(512) void ring_kernel(const MatmulParams p)
{
    constexpr int NW = 8, TM = FM * 16, TN = FN * 16, kStage = (TM + TN) * kStep, kLoads = 2 * (FM + FN);
    __shared__ __attribute__((aligned(16))) char smem[NW * STAGES * kStage];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Share share = xcd_share(p.tiles, blockIdx.x % kXcds);
    const int64_t id = share.first + blockIdx.x / kXcds, per = (int64_t)p.tiles_m * p.tiles_n;
    const int64_t batch = id / per;
    const int rest = (int)(id % per);
    const int64_t m0 = (int64_t)(rest % p.tiles_m) * TM, n0 = (int64_t)(rest / p.tiles_m) * TN;
    const int8_t *a = p.a + (batch * p.a_batch + m0) * p.K, *b = p.b + (batch * p.b_batch + n0) * p.K;
    const int rows_a = (int)(p.M - m0 < TM ? p.M - m0 : TM), rows_b = (int)(p.N - n0 < TN ? p.N - n0 : TN);
    RowLoads<2 * FM, DIRECT> loads_a;
    RowLoads<2 * FN, DIRECT> loads_b;
    loads_a.set(0, 8, rows_a, p.K);
    loads_b.set(0, 8, rows_b, p.K);

    const int each = (p.steps + NW - 1) / NW, from = wave * each;
    const int to = from + each < p.steps ? from + each : p.steps;
    char *mine = smem + wave * STAGES * kStage;
    const uint32_t lds = lds_address(mine);
    auto issue = [&](int step, int stage) {
        const uint32_t l = lds + stage * kStage;
        const int8_t *sa = a + (int64_t)step * kStep, *sb = b + (int64_t)step * kStep;
        const int left = p.K - step * kStep;
        if (left >= kStep) {
            loads_a.whole(l, 1024, sa);
            loads_b.whole(l + TM * kStep, 1024, sb);
        } else {
            loads_a.partial(l, 1024, sa, 0, 8, left);
            loads_b.partial(l + TM * kStep, 1024, sb, 0, 8, left);
        }
    };
    auto fetch = [&](int step) {
        const int left = p.K - step * kStep;
        loads_a.fetch(a + (int64_t)step * kStep, 0, 8, left, p.K);
        loads_b.fetch(b + (int64_t)step * kStep, 0, 8, left, p.K);
    };
    if constexpr (DIRECT) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            if (from + i < to)
                issue(from + i, i);
    } else if (from < to) {
        fetch(from);
    }
    // fragments: a lane holds 16 bytes of row lane % 16, quarter lane / 16
    const int fr = lane & 15, quarter = lane >> 4;
    i32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = i32x4{0, 0, 0, 0};
    int stage = 0;
    for (int s = from; s < to; ++s) {
        if constexpr (!DIRECT) {  // the next step is fetched while this one is worked on
            loads_a.put(mine, 1024);
            loads_b.put(mine + TM * kStep, 1024);
            if (s + 1 < to)
                fetch(s + 1);
        } else if (s + STAGES <= to) {  // arrived when only the younger stages' loads are pending
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads * (STAGES - 1)) : "memory");
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        }
        i32x4 fa[2][FM], fb[2][FN];
#pragma unroll
        for (int round = 0; round < 2; ++round) {
            const char *f = mine + stage * kStage + fr * kStep + place(fr, round * 4 + quarter) * 16;
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[round][i] = *(const i32x4 *)(f + i * 16 * kStep);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[round][j] = *(const i32x4 *)(f + (TM + j * 16) * kStep);
        }
        if constexpr (DIRECT) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the stage may be overwritten
            if (s + STAGES < to)
                issue(s + STAGES, stage);
        }
#pragma unroll
        for (int round = 0; round < 2; ++round)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[round][j], fa[round][i], acc[i][j], 0, 0, 0);
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
            *(i32x4 *)(mine + spread(i, j, quarter, fr)) = acc[i][j];
    __syncthreads();
    // four consecutive n of one m a thread
    using T = typename Elem<BF16>::T;
    const float *a_scale = p.a_scale + batch * p.a_batch + m0, *b_scale = p.b_scale + batch * p.b_batch + n0;
    T *out = (T *)p.out + (batch * p.M + m0) * p.N + n0;
    for (int i = threadIdx.x; i < TM * TN / 4; i += 64 * NW) {
        const int m = i / (TN / 4), n = i % (TN / 4) * 4;
        if (m >= rows_a || n >= rows_b)
            continue;
        const float sa = a_scale[m];
        const char *part = smem + spread(m / 16, n / 16, n % 16 / 4, m % 16);
        i32x4 sum = *(const i32x4 *)part;
#pragma unroll
        for (int w = 1; w < NW; ++w)
            sum += *(const i32x4 *)(part + w * kWaveBytes);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = (float)sum[e] * sa * b_scale[n + e < rows_b ? n + e : rows_b - 1];
        T *o = out + (int64_t)m * p.N + n;
        if (n + 4 <= rows_b) {
            if constexpr (BF16) {
                const u32x2 w = {cvt2(v[0], v[1]), cvt2(v[2], v[3])};
                __builtin_memcpy(o, &w, 8);
            } else {
                __builtin_memcpy(o, v, 16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (n + e < rows_b)
                    Elem<BF16>::store(o + e, v[e]);
        }
    }
}

// ---- choice --------------------------------------------------------------------------
//
// Which tile: the one whose time, by this model, is least, in us:
//   max(rounds * steps * alone, tiles / slots * steps * busy) + rounds * each + once
// rounds: output tiles a workgroup slot takes after one another; alone: a step
// of 128 bytes of the inner axis on an otherwise free card; busy: with every
// slot taken, where power and the shared caches hold the rate; each: a tile's
// end.  The constants are fitted to 520 shapes drawn from 8 x 16 to 16384 x 8192 with
// 64 to 8192 of the inner axis, each timed in every form; the form chosen takes
// 0.4 % more than the fastest on average, 1.5 % at the ninetieth percentile, and
// 16 % at the worst (2048 x 512 x 768: 7.4, 6.4).  Of two that tie, the one
// longer along n.  Both sides of some of the choices, in us:
//   8 x 5120 x 2048 x 2560   256 x 256 tiles 178, 128 x 128 217
//   4096 x 1536 x 768        256 x 256 tiles 13.3, 128 x 128 10.7
//   1024 x 2560 x 5120       128 x 128 tiles of two stages 31.8, of four 25.4, rings of 64 x 64 37.0
//   16384 x 2560 x 192       128 x 128 tiles of two stages 26.0, of four 30.8
//   1500 x 768 x 2560        128 x 128 tiles of four stages 15.3, 128 x 64 11.3, rings of 48 x 64 15.2
//   1024 x 2048 x 1024       128 x 128 tiles of four stages 8.8, 128 x 64 7.1
//   512 x 1536 x 768         128 x 128 tiles 7.0, rings of 64 x 64 6.0, of 64 x 48 5.5
//   256 x 2560 x 5120        rings of 64 x 64 12.8, of 64 x 48 11.9, of 48 x 64 11.4
//   64 x 2560 x 5120         rings of 32 x 64 9.6, of 32 x 32 7.3, of 16 x 32 10.0
//   64 x 5120 x 128          rings of 32 x 64 3.8, of 32 x 32 4.7, 128 x 128 tiles 4.8
//   2048 x 64 x 5120         rings of 32 x 32 7.5, of 16 x 32 6.7, of 32 x 16 9.0
//   16 x 2560 x 5120         rings of 32 x 32 6.7, of 16 x 32 6.2, of 16 x 16 5.3
enum Form { kTile256, kTile128, kTile128Deep, kTile64, kRing44, kRing34, kRing43, kRing24, kRing42, kRing22, kRing12, kRing21, kRing11, kForms };
struct FormCost {
    int tm, tn, slots;
    double alone, busy, each, once;
};
// A ring's loads bound it, alone or not.
constexpr FormCost ring_cost(int tm, int tn, bool direct)
{
    return direct ? FormCost{tm, tn, kCus, .00178 * (tm + tn), .00178 * (tm + tn), 1.04 + .00055 * tm * tn, 1.3}
                  : FormCost{tm, tn, kCus, .00281 * (tm + tn), .00281 * (tm + tn), 0.39 + .00088 * tm * tn, 2.1};
}
struct FormCosts {
    FormCost of[kForms];
};
constexpr FormCosts costs(FormCost tile256, FormCost tile128, FormCost tile128_deep, FormCost tile64, bool direct)
{
    return {{tile256, tile128, tile128_deep, tile64,
             ring_cost(64, 64, direct), ring_cost(48, 64, direct), ring_cost(64, 48, direct),
             ring_cost(32, 64, direct), ring_cost(64, 32, direct), ring_cost(32, 32, direct),
             ring_cost(16, 32, direct), ring_cost(32, 16, direct), ring_cost(16, 16, direct)}};
}
// By way of registers (fitted to 270 more shapes), of which 256 x 256 outputs leave none.
constexpr FormCosts kCosts[2] = {costs({}, {128, 128, 2 * kCus, 0.94, 1.69, 3.48, 3.85},
                                       {128, 128, kCus, 0.69, 0.90, 3.11, 2.92}, {128, 64, kCus, 0.66, 0.69, 2.17, 2.98}, false),
                                 costs({256, 256, kCus, 1.30, 1.50, 8.80, 1.30},
                                       {128, 128, 2 * kCus, 0.80, 1.15, 2.50, 2.50},
                                       {128, 128, kCus, 0.51, 0.69, 2.10, 2.60}, {128, 64, kCus, 0.41, 0.48, 1.75, 2.86}, true)};
constexpr int64_t kMostRingTiles = 1 << 16;  // of 512 threads

int64_t tiles_of(const FormCost &f, int64_t batch, int64_t M, int64_t N)
{
    return batch * ((M + f.tm - 1) / f.tm) * ((N + f.tn - 1) / f.tn);
}

Form choose(int64_t batch, int64_t M, int64_t N, int64_t K, bool direct)
{
    Form best = kTile128;
    double least = -1.;
    for (int f = direct ? kTile256 : kTile128; f < kForms; ++f) {
        const FormCost &c = kCosts[direct].of[f];
        const int64_t tiles = tiles_of(c, batch, M, N);
        if (f >= kRing44 && tiles > kMostRingTiles)
            continue;
        const double rounds = (double)((tiles + c.slots - 1) / c.slots), steps = (double)((K + kStep - 1) / kStep);
        const double alone = rounds * c.alone, busy = (double)tiles / c.slots * c.busy;
        const double cost = steps * (alone > busy ? alone : busy) + rounds * c.each + c.once;
        if (least < 0. || cost < least) {
            best = (Form)f;
            least = cost;
        }
    }
    return best;
}

template <int WM, int WN, int FM, int FN, int STAGES, bool DIRECT>
hipError_t tile(const MatmulParams &p, int slots, bool bf16, hipStream_t s)
{
    const dim3 grid((unsigned)(p.tiles < slots ? p.tiles : slots)), block(64 * WM * WN);
    // Rows that start at 64-byte boundaries are stored past the caches in whole
    // pieces of memory traffic (16384 x 5120 x 160: 40 us, 46 by the caches;
    // 16384 x 5152: 47 and 53); others leave pieces that a cache has to join
    // (16384 x 5128: 88 us past the caches, 56 by them; 5121: 99 and 58).
    const bool stream = (p.N * (bf16 ? 2 : 4)) % 64 == 0 && (uintptr_t)p.out % 64 == 0;
    if (bf16 && stream)
        tile_kernel<WM, WN, FM, FN, STAGES, DIRECT, true, true><<<grid, block, 0, s>>>(p);
    else if (bf16)
        tile_kernel<WM, WN, FM, FN, STAGES, DIRECT, true, false><<<grid, block, 0, s>>>(p);
    else if (stream)
        tile_kernel<WM, WN, FM, FN, STAGES, DIRECT, false, true><<<grid, block, 0, s>>>(p);
    else
        tile_kernel<WM, WN, FM, FN, STAGES, DIRECT, false, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <int FM, int FN, int STAGES> hipError_t ring(const MatmulParams &p, bool direct, bool bf16, hipStream_t s)
{
    const dim3 grid((unsigned)p.tiles), block(512);
    if (direct && bf16)
        ring_kernel<FM, FN, STAGES, true, true><<<grid, block, 0, s>>>(p);
    else if (direct)
        ring_kernel<FM, FN, STAGES, true, false><<<grid, block, 0, s>>>(p);
    else if (bf16)
        ring_kernel<FM, FN, 1, false, true><<<grid, block, 0, s>>>(p);
    else
        ring_kernel<FM, FN, 1, false, false><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

bool off16(const void *p) { return (uintptr_t)p % 16 != 0; }
bool is_direct(const Int8MatmulArgs &a) { return a.K % 16 == 0 && !off16(a.a) && !off16(a.b); }

}  // namespace

Int8MatmulForm int8_matmul_form(const Int8MatmulArgs &a)
{
    // one right operand for every batch: the batches' rows follow one another
    const bool joined = a.b_shared && !a.a_shared;
    Int8MatmulForm r{};
    r.batch = joined ? 1 : a.batch;
    r.M = joined ? a.batch * a.M : a.M;
    const bool direct = is_direct(a);
    r.form = choose(r.batch, r.M, a.N, a.K, direct);
    const FormCost &c = kCosts[direct].of[r.form];
    r.slots = c.slots;
    r.tile_m = c.tm;
    r.tile_n = c.tn;
    r.tiles = tiles_of(c, r.batch, r.M, a.N);
    return r;
}

hipError_t launch_int8_matmul(const Int8MatmulArgs &a, hipStream_t s)
{
    const bool direct = is_direct(a);
    const Int8MatmulForm f = int8_matmul_form(a);
    MatmulParams p{};
    p.a = a.a;
    p.b = a.b;
    p.a_scale = a.a_scale;
    p.b_scale = a.b_scale;
    p.out = a.out;
    p.M = f.M;
    p.N = a.N;
    p.K = (int)a.K;
    p.steps = a.K > 0 ? (int)((a.K + kStep - 1) / kStep) : 1;
    p.a_batch = a.a_shared ? 0 : f.M;
    p.b_batch = a.b_shared ? 0 : a.N;
    p.tiles_m = (int)((f.M + f.tile_m - 1) / f.tile_m);
    p.tiles_n = (int)((a.N + f.tile_n - 1) / f.tile_n);
    p.tiles = f.tiles;
    switch (f.form) {
    case kTile256: return tile<2, 4, 4, 2, 2, true>(p, f.slots, a.bf16, s);
    case kTile128:
        return direct ? tile<2, 2, 2, 2, 2, true>(p, f.slots, a.bf16, s) : tile<2, 2, 2, 2, 2, false>(p, f.slots, a.bf16, s);
    case kTile128Deep:
        return direct ? tile<4, 2, 1, 2, 4, true>(p, f.slots, a.bf16, s) : tile<4, 2, 1, 2, 4, false>(p, f.slots, a.bf16, s);
    case kTile64:
        return direct ? tile<4, 1, 1, 2, 3, true>(p, f.slots, a.bf16, s) : tile<4, 1, 1, 2, 3, false>(p, f.slots, a.bf16, s);
    case kRing44: return ring<4, 4, 1>(p, direct, a.bf16, s);
    case kRing43: return ring<4, 3, 1>(p, direct, a.bf16, s);
    case kRing34: return ring<3, 4, 1>(p, direct, a.bf16, s);
    case kRing42: return ring<4, 2, 1>(p, direct, a.bf16, s);
    case kRing24: return ring<2, 4, 1>(p, direct, a.bf16, s);
    case kRing22: return ring<2, 2, 2>(p, direct, a.bf16, s);
    case kRing12: return ring<1, 2, 2>(p, direct, a.bf16, s);
    case kRing21: return ring<2, 1, 2>(p, direct, a.bf16, s);
    default: return ring<1, 1, 2>(p, direct, a.bf16, s);
    }
}

}  // namespace mamba
