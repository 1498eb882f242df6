// pa_diff_decode_bf16.cu -- bf16 instantiations of the differential decode and its merge.
#include "pa_decode_mma.cuh"

namespace pa {
bool diff_decode_kernels_bf16(int head_dim, int group, KernelSet *ks)
{
    return diff_kernels<__nv_bfloat16>(head_dim, group, ks);
}
}  // namespace pa
