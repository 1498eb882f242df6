// pa_prefill.cu -- instantiations of the tcgen05 chunked-prefill kernel.
#include "pa_prefill.cuh"

namespace pa {

template <typename T, int D, bool DIFF>
static void prefill_entry(PrefillKernel *k)
{
    k->fn = reinterpret_cast<const void *>(&prefill_tc_kernel<T, D, DIFF>);
    k->threads = PrefillShape<D, DIFF>::THREADS;
    k->smem = PrefillShape<D, DIFF>::SMEM;
    k->plan_fn = reinterpret_cast<const void *>(&prefill_plan_kernel);
}

template <bool DIFF>
static bool pick(int dtype, int head_dim, PrefillKernel *k)
{
    const bool bf = dtype == PA_DTYPE_BF16;
    if (head_dim == 64)
        bf ? prefill_entry<__nv_bfloat16, 64, DIFF>(k) : prefill_entry<__half, 64, DIFF>(k);
    else if (head_dim == 128)
        bf ? prefill_entry<__nv_bfloat16, 128, DIFF>(k) : prefill_entry<__half, 128, DIFF>(k);
    else
        return false;
    return true;
}

bool prefill_kernel(int dtype, int head_dim, PrefillKernel *k)
{
    return pick<false>(dtype, head_dim, k);
}

bool diff_prefill_kernel(int dtype, int head_dim, PrefillKernel *k)
{
    return pick<true>(dtype, head_dim, k);
}

}  // namespace pa
