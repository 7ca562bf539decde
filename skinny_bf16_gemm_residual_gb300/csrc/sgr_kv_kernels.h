// sgr_kv_kernels.h -- the attention kernels' instances and their launch shapes.
// Those with masks (sinks, trees, a log-sum-exp) are instances of their own:
// in one, the code for masks cost calls without them 4 to 9% (registers of the
// walking warp and of the masked tiles: 19.8 against 21.7 us for 32 rows, 119
// against 127 for a chunk of a prompt).  They are compiled in a unit of their
// own (sgr_kv_masked.cu).
#pragma once

#include "sgr_kv_attn_few.cuh"
#include "sgr_kv_attn_rows.cuh"
#include "sgr_kv_mass.cuh"

namespace sgr {

using AttnFn = void (*)(const CUtensorMap, const CUtensorMap, const AttnParams);
using JoinFn = void (*)(const AttnParams);

struct AttnKernel {
  AttnFn fn;
  int smem, threads;
};

template <int D, int NT, bool kMasked>
AttnKernel attn_kernel_of() {
  return {kv_attn_kernel<D, NT, kMasked>, attn_smem_bytes<D, NT>(), AttnShape<D, NT>::kThreads};
}

// The kernel for row tiles of nt rows.
template <int D, bool kMasked>
AttnKernel attn_kernel_of(int nt) {
  switch (nt) {
    case 8: return attn_kernel_of<D, 8, kMasked>();
    case 16: return attn_kernel_of<D, 16, kMasked>();
    case 24: return attn_kernel_of<D, 24, kMasked>();
    case 32: return attn_kernel_of<D, 32, kMasked>();
    default: return {kv_attn_rows_kernel<D, kMasked>, rows_attn_smem_bytes<D>(), kRowsThreads};
  }
}

AttnKernel attn_kernel_masked(int dim, int nt);

// The sums of attention weights (sgr_kv_mass.cu).
using MassFn = void (*)(const CUtensorMap, const MassParams);
using MassJoinFn = void (*)(const MassParams);

struct MassKernel {
  MassFn fn;
  int smem, threads;
};

MassKernel mass_kernel(int dim, int nt);  // nt: 8, 16, 32 or kMassRows
MassJoinFn mass_join_kernel();            // of row tiles of kMassRows

}  // namespace sgr
