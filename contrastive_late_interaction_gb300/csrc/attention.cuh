// What the attention kernels share: the tapes' items and the element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cli_device.cuh"
#include "cli_internal.h"

namespace cli {
namespace attn {

// One item's rows on the tapes.  With shared queries q0 is 0 for every item,
// and its outputs start at o0.
struct Item {
    int q0, nq, k0, nk, o0;
    bool ok;
};

// Item i's rows, checked against the tapes' sizes: a malformed pair of offsets
// is reported and leaves the item without rows, so nothing is addressed
// through it.
__device__ __forceinline__ Item load_item(const AttentionLaunch &L, int i) {
    Item t;
    const uint64_t k0 = L.k_off[i], k1 = L.k_off[i + 1];
    uint64_t q0 = 0, q1 = static_cast<uint64_t>(L.query_rows);
    if (L.q_off) q0 = L.q_off[i], q1 = L.q_off[i + 1];
    t.ok = k0 <= k1 && k1 <= static_cast<uint64_t>(L.key_rows) && k1 - k0 <= static_cast<uint64_t>(L.max_k) &&
           q0 <= q1 && q1 <= static_cast<uint64_t>(L.query_rows) && q1 - q0 <= static_cast<uint64_t>(L.max_q) &&
           (i > 0 || (k0 == 0 && q0 == 0)) &&
           (i < L.items - 1 ||
            (k1 == static_cast<uint64_t>(L.key_rows) && q1 == static_cast<uint64_t>(L.query_rows)));
    if (!t.ok) {
        report(L.status, CLI_MALFORMED);
        t.q0 = t.nq = t.k0 = t.nk = t.o0 = 0;
        return t;
    }
    t.q0 = static_cast<int>(q0);
    t.nq = static_cast<int>(q1 - q0);
    t.k0 = static_cast<int>(k0);
    t.nk = static_cast<int>(k1 - k0);
    t.o0 = L.q_off ? t.q0 : i * L.query_rows;
    return t;
}

// Checks every item's offsets, the grid's threads sharing the items: kernels
// that reach items through their rows would not see all of a malformed tape.
__device__ __forceinline__ void check_items(const AttentionLaunch &L) {
    const long long threads = static_cast<long long>(gridDim.x) * gridDim.y * blockDim.x;
    for (long long i = (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
         i < L.items; i += threads)
        load_item(L, static_cast<int>(i));
}

}  // namespace attn
}  // namespace cli
