// Internal declarations of the operators around the scan (the residual RMS
// norm, the 8-bit quantiser, the 8-bit matrix product): shared by their host
// side (quant_api.cpp) and their kernels.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mamba {

// Longest row the norms and the token-major quantiser take: 1024 threads of
// four 8-element chunks hold it in registers.
constexpr int64_t kMaxNormWidth = 32768;

struct NormArgs {
    const void *x, *residual;  // [M, D]; residual NULL = none
    const float *weight;       // [D]; NULL = quantise x itself (no norm)
    void *out;                 // [M, D] of the I/O type, or int8
    float *scale;              // [M] (int8 output) or NULL
    void *residual_out;        // [M, D] or NULL
    int64_t M;
    int D;
    float eps;
    bool bf16, residual_bf16;
};
hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s);

struct NormBwdArgs {
    const void *dy, *h, *dres_out;  // [M, D]; dres_out NULL = zero
    const float *weight;
    void *dx, *dres;  // dres NULL = not returned
    float *dweight;   // [D]
    float *partials;  // [groups, D]
    int64_t M;
    int D;
    float eps;
    bool bf16, h_bf16;
};
// Groups of rows whose weight gradients are summed apart, one partial row each.
int64_t rms_norm_bwd_groups(int64_t M, int64_t D);
hipError_t launch_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s);

struct QuantChannelArgs {
    const void *x;  // [B, K, L]
    int8_t *q;      // [B, L, K]
    float *scale;   // [B, L]
    int64_t B, L, K;
    bool bf16;
};
hipError_t launch_quantize_channel_major(const QuantChannelArgs &a, hipStream_t s);

// Longest inner size of the 8-bit product: 2^14 (-128 times -128) per term
// stays below 2^31 over it, so the 32-bit sums are exact.
constexpr int64_t kMaxInner = 131071;

struct Int8MatmulArgs {
    const int8_t *a, *b;              // [batch or 1, M, K], [batch or 1, N, K]
    const float *a_scale, *b_scale;   // [batch or 1, M], [batch or 1, N]
    void *out;                        // [batch, M, N]
    int64_t batch, M, N, K;
    bool a_shared, b_shared, bf16;
};
hipError_t launch_int8_matmul(const Int8MatmulArgs &a, hipStream_t s);

// Which kernel a product takes (addresses count for their alignment only).
struct Int8MatmulForm {
    int form;           // number of the form
    int slots;          // workgroups that run at once; rings: one a tile
    int tile_m, tile_n; // outputs of a tile
    int64_t batch, M;   // of one product, batches of one right operand joined
    int64_t tiles;
};
Int8MatmulForm int8_matmul_form(const Int8MatmulArgs &a);

}  // namespace mamba
