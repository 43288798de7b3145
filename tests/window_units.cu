// The host side of the windowed attention (how a call is cut into units and what its
// workspace is sized for) as a library of its own, for test_window_units.py.
#include "window_attn.cu"

namespace uly {
int num_sms() { return 152; }
cudaError_t launch_window_fwd_bf16(const AttnShape &, const void *, const void *, const void *, void *, float *,
                                   cudaStream_t)
{
    return cudaErrorNotSupported;
}
cudaError_t launch_attn_bwd_bf16(const AttnShape &, const void *, const void *, const void *, const void *,
                                 const float *, const void *, void *, void *, void *, const BwdScratch &, cudaStream_t)
{
    return cudaErrorNotSupported;
}
cudaError_t launch_window_fwd_f32(const AttnShape &, const float *, const float *, const float *, float *, float *,
                                  cudaStream_t)
{
    return cudaErrorNotSupported;
}
cudaError_t launch_window_bwd_f32(const AttnShape &, const float *, const float *, const float *, const float *,
                                  const float *, const float *, float *, float *, float *, float *, cudaStream_t)
{
    return cudaErrorNotSupported;
}
}  // namespace uly

// {units, slots, joins, chunks} that the workspace has room for, and those of a call.
extern "C" void window_bounds(int64_t N, int64_t window, int64_t sinks, int num_docs, int tile, int64_t nprob,
                              int64_t *out)
{
    uly::unit_bounds(N, window, sinks, num_docs, tile, nprob, out[0], out[1], out[2], out[3]);
}

extern "C" void window_units(int64_t N, int window, int sinks, const int32_t *cu, int num_docs, int tile, int64_t nprob,
                             int64_t *out)
{
    const uly::Units r = uly::make_units(N, window, sinks, cu, num_docs, tile, nprob);
    out[0] = r.u.n_units;
    out[1] = r.u.slots;
    out[2] = r.u.n_joins;
    out[3] = r.u.n_chunks;
}

extern "C" size_t window_workspace(int64_t problems, int64_t N, int Hq, int Hkv, int64_t window, int64_t sinks,
                                   int num_docs, int esize)
{
    return uly::window_attn_workspace(problems, N, Hq, Hkv, 128, 1, window, sinks, num_docs, true, esize);
}
