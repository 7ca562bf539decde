// sgr_kv_mass.cu -- the instances of the kernels that sum attention weights.
#include "sgr_kv_kernels.h"

namespace sgr {

namespace {

template <int D, int NT>
MassKernel kernel_of() {
  return {kv_mass_kernel<D, NT>, mass_smem_bytes<D, NT>(), MassShape<D, NT>::kThreads};
}

template <int D>
MassKernel kernel_of(int nt) {
  switch (nt) {
    case 8: return kernel_of<D, 8>();
    case 16: return kernel_of<D, 16>();
    case 32: return kernel_of<D, 32>();
    default: return kernel_of<D, kMassRows>();
  }
}

}  // namespace

MassKernel mass_kernel(int dim, int nt) { return dim == 64 ? kernel_of<64>(nt) : kernel_of<128>(nt); }

MassJoinFn mass_join_kernel() { return kv_mass_join_kernel<kMassRows>; }

}  // namespace sgr
