// Host side of the C ABI of the gated linear recurrence: argument validation
// (before any HIP call) and launch.
#include "mamba_amd.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "gated_scan.h"
#include "host_check.h"

namespace {

// Rows (B * D) of a launch: four a workgroup of 256 threads, or fewer threads for
// a shorter row, below 2^32 threads in all.
constexpr int64_t kMaxGatedRows = int64_t(1) << 24;

int64_t chunks_of(int64_t L) { return (L + mamba::kGatedChunk - 1) / mamba::kGatedChunk; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// Maps of the parts that rows are split into.
size_t maps_bytes(int64_t B, int64_t D, int64_t L)
{
    const int parts = mamba::gated_parts(B * D, L).parts;
    return parts > 1 ? up256((size_t)(B * D * parts) * sizeof(float2)) : 0;
}
// Each row's and part's share of the parameters' gradients, where a channel has several.
size_t sums_bytes(int64_t B, int64_t D, int64_t L)
{
    const int parts = mamba::gated_parts(B * D, L).parts;
    return B * parts > 1 ? up256((size_t)(B * D * parts) * 3 * 4) : 0;
}

mamba_status gated_sizes(int64_t B, int64_t D, int64_t L, float c)
{
    if (!sizes_ok(B, D, L) || !(c >= 0.f) || std::isinf(c))
        return MAMBA_ERR_SHAPE;
    return B * D >= kMaxGatedRows || D >= kMaxGatedRows ? MAMBA_ERR_SHAPE : MAMBA_OK;  // D alone with B = 0
}

// What the forward call and the backward one read alike.
struct Inputs {
    const void *x, *r, *i, *z;
    const float *lam, *r_bias, *i_bias;
    const uint8_t *reset;
};
bool inputs_aligned(const Inputs &in, size_t es)
{
    return aligned(in.x, es) && aligned(in.r, es) && aligned(in.i, es) && aligned(in.z, es) && aligned(in.lam, 4) &&
           aligned(in.r_bias, 4) && aligned(in.i_bias, 4);
}

// No output overlaps an input, nor another output.
mamba_status apart(const Range *outs, int n_outs, const Range *ins, int n_ins)
{
    for (int o = 0; o < n_outs; ++o) {
        for (int k = 0; k < n_ins; ++k)
            if (overlap(outs[o], ins[k]))
                return MAMBA_ERR_ALIAS;
        for (int k = o + 1; k < n_outs; ++k)
            if (overlap(outs[o], outs[k]))
                return MAMBA_ERR_ALIAS;
    }
    return MAMBA_OK;
}

Range optional(const void *p, size_t bytes) { return rng(p, p ? bytes : 0); }

}  // namespace

extern "C" {

int64_t mamba_gated_scan_checkpoints(int64_t L) { return L > 0 && L <= kMaxElems ? chunks_of(L) : 0; }

size_t mamba_gated_scan_fwd_workspace_size(int64_t B, int64_t D, int64_t L)
{
    return gated_sizes(B, D, L, 0.f) == MAMBA_OK ? maps_bytes(B, D, L) : 0;
}

mamba_status mamba_gated_scan_fwd(const void *x, const void *r, const void *i, const float *lam, const float *r_bias,
                                  const float *i_bias, const void *z, const float *h0, const uint8_t *reset,
                                  void *y, float *h_last, float *checkpoints, void *workspace,
                                  size_t workspace_bytes, int64_t B, int64_t D, int64_t L, float c, mamba_dtype io,
                                  void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    const mamba_status sizes = gated_sizes(B, D, L, c);
    if (sizes != MAMBA_OK)
        return sizes;
    const int64_t rows = B * D;
    if (rows == 0 || (L == 0 && !h_last))
        return MAMBA_OK;
    if (!lam || (L > 0 && (!x || !r || !i || !y)))
        return MAMBA_ERR_NULL;
    const size_t es = esize(io), n = (size_t)(rows * L) * es, per_d = (size_t)D * 4;
    const Inputs in{x, r, i, z, lam, r_bias, i_bias, reset};
    if (!inputs_aligned(in, es) || !aligned(h0, 4) || !aligned(y, es) || !aligned(h_last, 4) ||
        !aligned(checkpoints, 4))
        return MAMBA_ERR_ALIGN;
    const size_t need = maps_bytes(B, D, L);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return MAMBA_ERR_WORKSPACE;
    const Range ins[] = {rng(x, n), rng(r, n), rng(i, n), optional(z, n), rng(lam, per_d), optional(r_bias, per_d),
                         optional(i_bias, per_d), optional(h0, (size_t)rows * 4),
                         optional(reset, (size_t)(B * L))};
    const Range outs[] = {rng(y, n), optional(h_last, (size_t)rows * 4),
                          optional(checkpoints, (size_t)(rows * chunks_of(L)) * 4), rng(workspace, need)};
    mamba_status st = apart(outs, 4, ins, 9);
    if (st != MAMBA_OK)
        return st;
    st = device_ok();
    if (st != MAMBA_OK)
        return st;
    const mamba::GatedParts split = mamba::gated_parts(rows, L);
    mamba::GatedScanArgs a{x, r, i, z, lam, r_bias, i_bias, h0, reset, y, h_last, checkpoints,
                           c, B, D, L, io == MAMBA_BF16, (float2 *)workspace, split.steps, split.parts};
    return launched(mamba::launch_gated_scan_fwd(a, (hipStream_t)stream));
}

size_t mamba_gated_scan_bwd_workspace_size(int64_t B, int64_t D, int64_t L, int with_checkpoints)
{
    if (gated_sizes(B, D, L, 0.f) != MAMBA_OK)
        return 0;
    const size_t rows = (size_t)(B * D);
    return sums_bytes(B, D, L) + maps_bytes(B, D, L) + (with_checkpoints ? 0 : up256(rows * (size_t)chunks_of(L) * 4));
}

mamba_status mamba_gated_scan_bwd(const void *x, const void *r, const void *i, const float *lam, const float *r_bias,
                                  const float *i_bias, const void *z, const float *h0, const uint8_t *reset,
                                  const float *checkpoints, const void *dout, const float *dh_last, void *dx,
                                  void *dr, void *di, void *dz, float *dlam, float *dr_bias, float *di_bias,
                                  float *dh0, void *workspace, size_t workspace_bytes, int64_t B, int64_t D,
                                  int64_t L, float c, mamba_dtype io, void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    const mamba_status sizes = gated_sizes(B, D, L, c);
    if (sizes != MAMBA_OK)
        return sizes;
    if (D == 0)
        return MAMBA_OK;
    const int64_t rows = B * D;
    if (!lam || !dlam || !dr_bias || !di_bias || (rows > 0 && !dh0))
        return MAMBA_ERR_NULL;
    if (rows * L > 0 && (!x || !r || !i || !dout || !dx || !dr || !di || (z && !dz)))
        return MAMBA_ERR_NULL;
    if (dz && !z)
        return MAMBA_ERR_UNSUPPORTED;
    const size_t es = esize(io), n = (size_t)(rows * L) * es, per_d = (size_t)D * 4, per_row = (size_t)rows * 4;
    const Inputs in{x, r, i, z, lam, r_bias, i_bias, reset};
    if (!inputs_aligned(in, es) || !aligned(h0, 4) || !aligned(checkpoints, 4) || !aligned(dout, es) ||
        !aligned(dh_last, 4) || !aligned(dx, es) || !aligned(dr, es) || !aligned(di, es) || !aligned(dz, es) ||
        !aligned(dlam, 4) || !aligned(dr_bias, 4) || !aligned(di_bias, 4) || !aligned(dh0, 4))
        return MAMBA_ERR_ALIGN;
    const size_t kept = (size_t)(rows * chunks_of(L)) * 4;
    const size_t need = mamba_gated_scan_bwd_workspace_size(B, D, L, checkpoints != nullptr);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return MAMBA_ERR_WORKSPACE;
    const Range ins[] = {rng(x, n), rng(r, n), rng(i, n), optional(z, n), rng(lam, per_d), optional(r_bias, per_d),
                         optional(i_bias, per_d), optional(h0, per_row), optional(reset, (size_t)(B * L)),
                         optional(checkpoints, kept), rng(dout, n), optional(dh_last, per_row)};
    const Range outs[] = {rng(dx, n), rng(dr, n), rng(di, n), optional(dz, n), rng(dlam, per_d), rng(dr_bias, per_d),
                          rng(di_bias, per_d), optional(dh0, per_row), rng(workspace, need)};
    mamba_status st = apart(outs, 9, ins, 12);
    if (st != MAMBA_OK)
        return st;
    st = device_ok();
    if (st != MAMBA_OK)
        return st;
    mamba::GatedScanBwdArgs a{};
    const mamba::GatedParts split = mamba::gated_parts(rows, L);
    unsigned char *ws = (unsigned char *)workspace, *maps = ws + sums_bytes(B, D, L);
    a.f = mamba::GatedScanArgs{x, r, i, z, lam, r_bias, i_bias, h0, reset, nullptr, nullptr,
                               const_cast<float *>(checkpoints), c, B, D, L, io == MAMBA_BF16, (float2 *)maps,
                               split.steps, split.parts};
    if (!checkpoints && rows * L > 0) {  // the forward pass again, for its states alone
        a.f.checkpoints = (float *)(maps + maps_bytes(B, D, L));
        st = launched(mamba::launch_gated_scan_fwd(a.f, (hipStream_t)stream));
        if (st != MAMBA_OK)
            return st;
    }
    a.dout = dout;
    a.dh_last = dh_last;
    a.dx = dx;
    a.dr = dr;
    a.di = di;
    a.dz = dz;
    a.dlam = dlam;
    a.dr_bias = dr_bias;
    a.di_bias = di_bias;
    a.dh0 = dh0;
    a.partials = (float *)workspace;
    return launched(mamba::launch_gated_scan_bwd(a, (hipStream_t)stream));
}

mamba_status mamba_gated_state_update(const float *h, float *h_out, const void *x, const void *r, const void *i,
                                      const float *lam, const float *r_bias, const float *i_bias, const void *z,
                                      void *y, int64_t B, int64_t D, float c, mamba_dtype io, void *stream)
{
    if (!valid_dtype(io))
        return MAMBA_ERR_DTYPE;
    if (!sizes_ok(B, D, 1) || !(c >= 0.f) || std::isinf(c) || B * D >= int64_t(1) << 31)
        return MAMBA_ERR_SHAPE;
    const int64_t rows = B * D;
    if (rows == 0)
        return MAMBA_OK;
    if (!h || !h_out || !x || !r || !i || !lam || !y)
        return MAMBA_ERR_NULL;
    const size_t es = esize(io), n = (size_t)rows * es, per_d = (size_t)D * 4, states = (size_t)rows * 4;
    const Inputs in{x, r, i, z, lam, r_bias, i_bias, nullptr};
    if (!inputs_aligned(in, es) || !aligned(h, 4) || !aligned(h_out, 4) || !aligned(y, es))
        return MAMBA_ERR_ALIGN;
    // the state may be updated in place, as the very same buffer
    const Range ins[] = {rng(x, n), rng(r, n), rng(i, n), optional(z, n), rng(lam, per_d), optional(r_bias, per_d),
                         optional(i_bias, per_d), rng(h, h_out == h ? 0 : states)};
    const Range outs[] = {rng(y, n), rng(h_out, states)};
    mamba_status st = apart(outs, 2, ins, 8);
    if (st != MAMBA_OK)
        return st;
    st = device_ok();
    if (st != MAMBA_OK)
        return st;
    mamba::GatedStepArgs a{x, r, i, z, lam, r_bias, i_bias, h, h_out, y, c, B, D, io == MAMBA_BF16};
    return launched(mamba::launch_gated_step(a, (hipStream_t)stream));
}

}  // extern "C"
