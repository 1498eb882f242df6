// pa_prefill_plan.cuh -- how a prefill block finds its work in the work order
// that prefill_plan_kernel leaves (PrefillParams::plan).
#pragma once

#include "pa_device.cuh"
#include "pa_prefill_abi.h"

namespace pa {

// The (sequence, query tile, kv head) of block b under the work order;
// false past the end of the order.
__device__ __forceinline__ bool plan_block(const PrefillParams &p, int b, int &s, int &tile,
                                           int &h)
{
    const int Hkv = p.num_kv_heads;
    const int k = b / Hkv;
    if (k >= *p.plan_count)
        return false;
    uint32_t e = p.plan[k];
    if (*p.plan_by_seq) {
        const int s0 = (int)(e >> 16);
        const int st = p.plan_seq_start[s0], nq = p.plan_seq_nq[s0];
        const int local = b - Hkv * st;
        h = local / nq;
        e = p.plan[st + local % nq];
    } else {
        h = b % Hkv;
    }
    s = (int)(e >> 16);
    tile = (int)(e & 0xffffu);
    return true;
}

}  // namespace pa
