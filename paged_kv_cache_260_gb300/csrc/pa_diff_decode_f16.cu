// pa_diff_decode_f16.cu -- fp16 instantiations of the differential decode and its merge.
#include "pa_decode_mma.cuh"

namespace pa {
bool diff_decode_kernels_f16(int head_dim, int group, KernelSet *ks)
{
    return diff_kernels<__half>(head_dim, group, ks);
}
}  // namespace pa
