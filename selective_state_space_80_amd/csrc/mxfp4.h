// Internal declarations of the microscaled 4-bit format (quantiser, the way back,
// matrix product): shared by their host side (mxfp4_api.cpp) and their kernels.
// Not part of the public C ABI.
//
// A row of K elements is filled up with zeros to whole groups of 256: 128 bytes, a
// cache line, and 8 scales.  Packed rows lie one behind the other; scales lie by
// group, [groups, rows, 8], so that a product's step of one group takes the scales
// of neighbouring rows from neighbouring addresses.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

constexpr int kMxGroup = 256;        // elements of a group
constexpr int kMxGroupBytes = 128;   // packed
constexpr int kMxScales = 8;         // scales of a group: one for every 32 elements
constexpr int64_t kMaxMxInner = int64_t(1) << 23;

constexpr int64_t mx_groups(int64_t K) { return (K + kMxGroup - 1) / kMxGroup; }

struct MxQuantArgs {
    const void *x;   // [rows, K] of the I/O type; channel-major [B, K, L]
    uint8_t *q;      // [rows, groups * 128]
    uint8_t *scale;  // [groups, rows, 8]
    int64_t B, L, K; // rows = B * L
    bool bf16;
};
hipError_t launch_quantize_mxfp4(const MxQuantArgs &a, hipStream_t s);
hipError_t launch_quantize_mxfp4_channel_major(const MxQuantArgs &a, hipStream_t s);

struct MxDequantArgs {
    const uint8_t *q, *scale;
    void *out;       // [rows, K]
    int64_t rows, K;
    bool bf16;
};
hipError_t launch_dequantize_mxfp4(const MxDequantArgs &a, hipStream_t s);

struct MxMatmulArgs {
    const uint8_t *a, *a_scale;  // [batch or 1, M, groups * 128], [groups, batch or 1, M, 8]
    const uint8_t *b, *b_scale;  // of N rows
    void *out;                   // [batch, M, N]
    int64_t batch, M, N, groups;
    bool a_shared, b_shared, bf16;
};
// Which kernel a product takes.
struct MxMatmulForm {
    int form;           // number of the form
    int slots;          // workgroups that run at once; rings: one a tile
    int tile_m, tile_n; // outputs of a tile
    int64_t batch, M;   // of one product, batches of one right operand joined
    int64_t tiles;
};
MxMatmulForm mxfp4_matmul_form(const MxMatmulArgs &a);
hipError_t launch_mxfp4_matmul(const MxMatmulArgs &a, hipStream_t s);

}  // namespace mamba
