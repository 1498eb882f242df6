// pa_mass_decode_bf16.cu -- bf16 instantiations of the decode that leaves its scores.
#include "pa_decode_mma.cuh"

namespace pa {
bool mass_decode_kernels_bf16(int head_dim, int group, KernelSet *ks)
{
    return mass_kernels<__nv_bfloat16>(head_dim, group, ks);
}
}  // namespace pa
