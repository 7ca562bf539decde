// sgr_kv_masked.cu -- the attention kernels with masks.
#include "sgr_kv_kernels.h"

namespace sgr {

AttnKernel attn_kernel_masked(int dim, int nt) {
  return dim == 64 ? attn_kernel_of<64, true>(nt) : attn_kernel_of<128, true>(nt);
}

}  // namespace sgr
