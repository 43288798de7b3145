// The norms around a block (residual_norm.cuh): how a call is laid over the GPU, its
// workspace, and the bf16 kernels (residual_norm_f32.cu: the fp32 ones).
#include "residual_norm.cuh"

namespace uly {
namespace {

ResidualNormPlan plan_for(int64_t T, int64_t run, int D, int esize, bool bwd)
{
    ResidualNormPlan q;
    const int row_bytes = D * esize, nvec = row_bytes / 16, tensors = bwd ? 4 : 2;
    // The ring: about 100 KB (backward 120).  More on their way do not help and are
    // shared out unevenly: with 200 KB the first blocks of a 203 us call ended
    // after 170, the last after 235; with 60 KB all of them after 222.
    const int64_t room = (bwd ? 122 : 102) * 1024;
    q.lanes = 32;
    while (q.lanes > 1 && q.lanes / 2 >= nvec)
        q.lanes /= 2;
    // A slot: a row, or as many short ones as leave two slots for each of 15 warps,
    // but no more than every warp has some of.
    const int64_t share = (T + static_cast<int64_t>(num_sms()) * kMaxWarps - 1) / (num_sms() * kMaxWarps);
    const int64_t fit = room / (2 * kMaxWarps * tensors) / row_bytes;
    q.slot_rows = static_cast<int>(
        std::min(std::min<int64_t>(run, kMaxRows), std::max<int64_t>(1, std::min<int64_t>(share, fit))));
    const int64_t slot = static_cast<int64_t>(tensors) * q.slot_rows * row_bytes;
    // Groups of two slots each, and the warps among them; a thread has up to 4 chunks
    // of a row (backward 2, whose sums stay in registers) unless 15 warps are too few.
    const int64_t slots = std::max<int64_t>(1, room / slot);
    q.groups = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxWarps, slots / 2)));
    const int cap = bwd ? 2 : 4;
    q.warps = std::max(kMaxWarps / q.groups, std::min(kMaxWarps, (nvec + 32 * cap - 1) / (32 * cap)));
    q.chunks = (nvec + 32 * q.warps - 1) / (32 * q.warps);
    q.warps = (nvec + 32 * q.chunks - 1) / (32 * q.chunks);
    q.groups = std::min(q.groups, kMaxWarps / q.warps);
    q.parts = q.groups * (32 / q.lanes) > 1 ? q.groups * (32 / q.lanes) : 0;
    q.threads = (q.groups * q.warps + 1) * 32;
    // every group its own slots
    const size_t most = static_cast<size_t>(227) * 1024;
    auto bytes = [&](int own) {
        const int n = own * q.groups;
        return Smem::fixed(D, row_bytes, bwd ? q.parts : 0, bwd ? n : 0) + static_cast<size_t>(n) * slot;
    };
    int own = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>(slots, kMaxSlots) / q.groups));
    while (own > 1 && (own * q.groups > kMaxSlots || bytes(own) > most))
        --own;
    q.slots = own * q.groups;
    q.smem = bytes(own);
    const int64_t units = (T + q.slot_rows - 1) / q.slot_rows;
    q.blocks = static_cast<int>(std::min<int64_t>(units, num_sms()));
    q.block_rows = static_cast<int>((T + q.blocks - 1) / q.blocks);
    if (run < T)  // runs of rows: none of the blocks is empty
        q.blocks = static_cast<int>((T + q.block_rows - 1) / q.block_rows);
    return q;
}

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// Bytes of the blocks' sums: those of w1, then those of the gates' runs.
void partial_bytes(const ResidualNormPlan &q, int64_t T, int64_t run, int D, size_t &one, size_t &gates)
{
    const int64_t runs = (T + run - 1) / run;
    one = up(static_cast<size_t>(q.blocks) * D * sizeof(float));
    gates = up(static_cast<size_t>(q.blocks + runs) * D * sizeof(float));
}

}  // namespace

size_t residual_norm_workspace(int64_t T, int64_t Np, int D)
{
    // the largest of the element types, gates shared or a sequence's own; a type whose
    // rows are no multiple of 16 bytes, which a call refuses, has no plan
    size_t most = 0;
    for (int es = 2; es <= 4; es += 2)
        for (const int64_t run : {T, Np}) {
            if (D * es > 32768 || D * es % 16 != 0)
                continue;
            size_t one, gates;
            partial_bytes(plan_for(T, run, D, es, true), T, run, D, one, gates);
            most = std::max(most, one + gates);
        }
    return most;
}

cudaError_t launch_residual_norm(ResidualNormParams &p, bool bwd, int esize, void *workspace, cudaStream_t s)
{
    const ResidualNormPlan q = plan_for(p.T, p.run, p.D, esize, bwd);
    p.warps = q.warps;
    p.lanes = q.lanes;
    p.groups = q.groups;
    p.parts = bwd ? q.parts : 0;
    p.slot_rows = q.slot_rows;
    p.slots = q.slots;
    p.block_rows = q.block_rows;
    p.w = wait_cfg();
    if (bwd && workspace) {
        size_t one, gates;
        partial_bytes(q, p.T, p.run, p.D, one, gates);
        p.part1_elems = static_cast<int64_t>(one / sizeof(float));
        p.partA_elems = static_cast<int64_t>(gates / sizeof(float));
        p.part1 = p.dw1 ? static_cast<float *>(workspace) : nullptr;
        p.partA = p.dw2 || p.dgate ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + one) : nullptr;
    }
    return esize == 2 ? launch_residual_norm_typed<uint16_t>(p, q, bwd, s) : launch_residual_norm_f32(p, q, bwd, s);
}

}  // namespace uly
