// pa_mass_decode_f16.cu -- f16 instantiations of the decode that leaves its scores.
#include "pa_decode_mma.cuh"

namespace pa {
bool mass_decode_kernels_f16(int head_dim, int group, KernelSet *ks)
{
    return mass_kernels<__half>(head_dim, group, ks);
}
}  // namespace pa
