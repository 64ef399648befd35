// Internal declarations of the gated linear recurrence: shared by its host side
// (gated_scan_api.cpp) and its kernels.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

// Steps between the states that the forward call keeps for the backward one:
// what a wave takes at once, 8 steps a lane.
constexpr int kGatedChunk = 512;

struct GatedScanArgs {
    const void *x, *r, *i, *z;                 // [B, D, L] of the I/O type; z NULL = no gate
    const float *lam, *r_bias, *i_bias, *h0;   // [D], [D], [D], [B, D]; the last three may be NULL
    const uint8_t *reset;                      // [B, L] or NULL
    void *y;                                   // [B, D, L], or NULL (checkpoints only)
    float *h_last, *checkpoints;               // [B, D], [B, D, ceil(L / kGatedChunk)]; may be NULL
    float c;
    int64_t B, D, L;
    bool bf16;
    // rows split into parts (gated_parts), whose maps are worked out first
    float2 *maps;        // [B, D, parts]
    int64_t part_steps;
    int parts;
};

// Few rows of many steps: parts of a row that different workgroups take, at most 64
// (a wave joins their maps), each of whole chunks.  One part: no split.
struct GatedParts {
    int parts;
    int64_t steps;  // of a part
};
GatedParts gated_parts(int64_t rows, int64_t L);
hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t s);

struct GatedScanBwdArgs {
    GatedScanArgs f;                // of the forward call (y, h_last unused); checkpoints is an input
    const void *dout;               // [B, D, L]
    const float *dh_last;           // [B, D] or NULL
    void *dx, *dr, *di, *dz;        // [B, D, L]; dz NULL without z
    float *dlam, *dr_bias, *di_bias, *dh0;  // [D], [D], [D], [B, D]
    float *partials;                // [3, parts, B, D]; unused with one row a channel
};
hipError_t launch_gated_scan_bwd(const GatedScanBwdArgs &a, hipStream_t s);

struct GatedStepArgs {
    const void *x, *r, *i, *z;                // [B, D]
    const float *lam, *r_bias, *i_bias, *h;   // h [B, D]
    float *h_out;                             // [B, D], may be h itself
    void *y;
    float c;
    int64_t B, D;
    bool bf16;
};
hipError_t launch_gated_step(const GatedStepArgs &a, hipStream_t s);

}  // namespace mamba
