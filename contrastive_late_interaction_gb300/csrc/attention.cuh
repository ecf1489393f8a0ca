// What the attention kernels share: the tapes' items, the element types and
// the pieces of their tensor-core pipelines.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cli_device.cuh"
#include "cli_internal.h"
#include "launch.cuh"

namespace cli {
namespace attn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// Checks every item's offsets, `threads` threads of the grid sharing them:
// kernels that reach items through their rows would not see all of a
// malformed tape.
__device__ __forceinline__ void check_items(const AttentionLaunch &L, long long thread, long long threads) {
    for (long long i = thread; i < L.items; i += threads) load_item(L, static_cast<int>(i));
}

// Rows of a tape are worked on in blocks of `span` rows that start at each
// item's first row.  Block slot x belongs to the item i with
//     first(i) <= x < first(i + 1),   first(i) = offsets[i] / span + i,
// and is its block x - first(i): an item of n rows has ceil(n / span) blocks
// and at least that many slots, since floor((o + n) / span) - floor(o / span)
// + 1 >= ceil(n / span); at most one slot per item stays empty.  So the slots
// (rows / span + items of them) need no table and no scan: a search over the
// offsets finds the item.  A warp searches 32 ways:
__device__ __forceinline__ int find_item(const uint64_t *off, int items, unsigned span, long long x, int lane) {
    int lo = 0, n = items;   // the item is one of lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < n && static_cast<long long>(off[at] / span) + at <= x;
        const unsigned hits = __ballot_sync(0xffffffffu, le);
        const int k = hits ? 31 - __clz(hits) : 0;
        const int left = n - k * step;
        lo += k * step;
        n = left < step ? left : step;
    }
    return lo;
}

// A thread on its own, in halves.
__device__ __forceinline__ int find_item(const uint64_t *off, int items, unsigned span, long long x) {
    int lo = 0, hi = items;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<long long>(off[mid] / span) + mid <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Block `x` of a tape cut into blocks of `span` rows, or of shared queries
// (off NULL) with `per_item` blocks an item: its item and the row it starts
// at; false where the slot is empty.  `known` is the item where the warp has
// searched for it, and -1 where it has not.
__device__ __forceinline__ bool find_block(const AttentionLaunch &L, const uint64_t *off, unsigned span, int per_item,
                                           bool of_keys, long long x, Item &t, int &r0, int known = -1) {
    int i;
    long long block;
    if (off) {
        i = known >= 0 ? known : find_item(off, L.items, span, x);
        block = x - (static_cast<long long>(off[i] / span) + i);
    } else {
        i = static_cast<int>(x / per_item);
        block = x - static_cast<long long>(i) * per_item;
    }
    t = load_item(L, i);
    const long long at = block * span;
    r0 = static_cast<int>(at);
    return t.ok && block >= 0 && at < (of_keys ? t.nk : t.nq);
}

// A wait of a whole warp, whose lanes come out of it together and agree on
// whether it was given up.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status)) != 0;
}

// The tensor-core kernels hand out their blocks from a counter, a batch at a
// time: items differ in length, and every other slot may be empty.  A warp
// looks up a batch at once, one block a lane, so that the search costs each
// block little, and enough batches are left to even out the CTAs.
__device__ __forceinline__ int batch_of(long long tiles) {
    const long long b = tiles / (static_cast<long long>(gridDim.x) * 8);
    return b < 1 ? 1 : b > 32 ? 32 : static_cast<int>(b);
}

constexpr size_t kCounterBytes = 256;   // at the start of the workspace: the counters, and from word kBoundsAt on bounds
constexpr int kBoundsAt = 16;

// The first kernel of a call: the status, the counters and the bounds start at 0.
static __global__ void begin_kernel(int32_t *status, unsigned long long *counters) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) *status = 0;
    if (threadIdx.x < kCounterBytes / 8) counters[threadIdx.x] = 0;
}

template <typename T> struct Type;
template <> struct Type<__nv_bfloat16> {
    static constexpr bool bf16 = true;
    static constexpr uint16_t one = 0x3F80, infinity = 0x7F80;
    static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
};
template <> struct Type<__half> {
    static constexpr bool bf16 = false;
    static constexpr uint16_t one = 0x3C00, infinity = 0x7C00;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
};

// fp16 as the type of P and dS, whose products' gradients may be of any size:
// P goes in times 2^14, and dS times a power of two that brings it below 2^15,
// so that neither leaves the type's normal range downwards while the other end
// holds (in their own size dQ and dK had 6 times the error at output gradients
// of 0.001, and infinities at 10^5).  In bf16 both stay as they are.
template <typename T> __host__ __device__ constexpr float weight_shift() { return Type<T>::bf16 ? 0.0f : 14.0f; }
template <typename T> __host__ __device__ constexpr float weight_unit() { return Type<T>::bf16 ? 1.0f : 1.0f / 16384.0f; }

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// The e of a positive normal number's 2^e <= x < 2^(e + 1).
__device__ __forceinline__ int exponent_of(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Word w of the kept-states mask of a block of which the first n are there.
__device__ __forceinline__ uint32_t first_bits(int n, int w) {
    const int left = n - 32 * w;
    return left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
}

// The kept ones of the n states (at most 128) from k0, as bits.  One warp.
__device__ __forceinline__ void kept_bits(const AttentionLaunch &L, int k0, int n, int lane, uint32_t (&keep)[4]) {
    uint8_t byte[4];
    if (L.key_mask) {
#pragma unroll
        for (int w = 0; w < 4; ++w) byte[w] = 32 * w + lane < n ? L.key_mask[k0 + 32 * w + lane] : 0;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) keep[w] = L.key_mask ? __ballot_sync(0xffffffffu, byte[w] != 0) : first_bits(n, w);
}

__device__ __forceinline__ uint32_t round16(int n) { return static_cast<uint32_t>((n + 15) & ~15); }

// Shared-memory tiles: rows of 64 elements (128 bytes, 128-byte swizzle), one
// box of kBoxBytes per 64 elements of the head.
constexpr uint32_t kTileRows = 128;
constexpr uint32_t kBoxBytes = kTileRows * 128;

// Descriptors of a tile: rows of heads as a K-major operand, and as the
// MN-major operand of a product that sums over the rows.  The address field
// counts 16 bytes, so a step within a tile is an addition to the descriptor.
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile) { return sdesc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_sum(uint32_t tile) { return sdesc_sw128(tile, kBoxBytes, 1024); }
constexpr uint64_t desc_bytes(uint32_t bytes) { return bytes >> 4; }

// Products are issued by one thread, but by code that the whole warp runs
// along, with the thread chosen by elect.sync: the compiler then keeps the
// descriptors in uniform registers, where the instruction wants them, and an
// instruction or two go out per product.  Eight products of 128 x 128 x 16
// (64 cycles each) took 1160 cycles from a branch of lane 0, 940 predicated on
// lane 0, and take 680 predicated on the elected thread.
__device__ __forceinline__ uint32_t elected() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ void issue_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p, q;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void issue_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p, q;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
        "}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
// Arrives on `bar` when the products issued so far are complete.
__device__ __forceinline__ void issue_commit(uint32_t leader, uint64_t *bar) {
    asm volatile(
        "{\n"
        " .reg .pred q;\n"
        " setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
        "}\n" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}

// Descriptor of a K-major operand of 16 elements a row without a swizzle: 8
// rows of 16 bytes are 128 bytes in a row, 8-row groups follow one another,
// the second 8 elements lie 2 KB on.
constexpr uint32_t kColumnBytes = 4096;
__device__ __forceinline__ uint64_t desc_column(uint32_t at) {
    return static_cast<uint64_t>((at & 0x3FFFFu) >> 4) | static_cast<uint64_t>(2048 >> 4) << 16 |
           static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}

// D = A B^T over `steps` times 16 elements of the heads.  The usual count has
// code without conditions: one before each product costs as much as the product.
template <int BOXES>
__device__ __forceinline__ void mma_rows(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int steps) {
    auto step = [&](int k) {
        const uint64_t at = desc_bytes((k >> 2) * kBoxBytes + (k & 3) * 32);
        issue_ss(leader, d, a + at, b + at, idesc, k != 0);
    };
    if (steps == 4 * BOXES) {
#pragma unroll
        for (int k = 0; k < 4 * BOXES; ++k) step(k);
    } else {
#pragma unroll 1
        for (int k = 0; k < steps; ++k) step(k);
    }
}

// D (+)= A B over `rows` rows of B, at most 16 STEPS; A in TMEM (16-bit pairs), B a tile
// of rows of heads.
template <int STEPS>
__device__ __forceinline__ void mma_pairs(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, int rows,
                                          bool accumulate) {
    const uint32_t first = accumulate;
    if (rows > 16 * (STEPS - 1)) {
        issue_ts(leader, d, a, b, idesc, first);
#pragma unroll
        for (int k = 1; k < STEPS; ++k) issue_ts(leader, d, a + k * 8, b + desc_bytes(k * 2048), idesc, 1);
    } else {
#pragma unroll 1
        for (int k = 0; 16 * k < rows; ++k)
            issue_ts(leader, d, a + k * 8, b + desc_bytes(k * 2048), idesc, k != 0 ? 1 : first);
    }
}

// 32 bytes to global memory, in one request where the address allows it.
__device__ __forceinline__ void store_32(void *p, bool wide, const uint32_t (&v)[8]) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// A row of `dim` sums (a multiple of 8) at `sums` in TMEM, times `scale`, as
// 16-bit values to `out`; zeros where `zero`, or where the warp has no sums.  A thread writes its own row, whole
// sectors at a time; going through shared memory for contiguous requests was
// no faster, since the products' operands keep that busy.
template <typename T>
__device__ __forceinline__ void store_sums(uint32_t sums, int dim, float scale, bool warp_has, bool zero, bool mine, T *out) {
    const bool wide = reinterpret_cast<uintptr_t>(out) % 32 == 0;
#pragma unroll 1
    for (int x = 0; x < dim; x += 16) {
        uint32_t r[16], v[8];
        if (warp_has) {   // the same for the whole warp, as the load demands
            tmem_ld16_async(sums + x, r);
            tmem_wait_ld();
            tmem_regs_ready_n(r);
        }
        if (mine) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = warp_has && !zero ? Type<T>::pack(__uint_as_float(r[2 * i]) * scale, __uint_as_float(r[2 * i + 1]) * scale)
                                        : 0u;
            if (x + 16 <= dim)
                store_32(out + x, wide, v);
            else
                *reinterpret_cast<uint4 *>(out + x) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        __syncwarp();   // the loads above are the whole warp's
    }
}

// The same as 32-bit sums; `out` on 32 bytes.
__device__ __forceinline__ void store_partials(uint32_t sums, int dim, float scale, bool warp_has, bool mine, float *out) {
#pragma unroll 1
    for (int x = 0; x < dim; x += 8) {
        uint32_t r[8] = {};
        if (warp_has) {
            tmem_ld8_async(sums + x, r);
            tmem_wait_ld();
            tmem_regs_ready_n(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * scale);
        }
        if (mine) store_32(out + x, true, r);
        __syncwarp();
    }
}

// The cuts go by the 152 SMs of a GB300 rather than by the device's own count, so that the sizers, which are asked without a
// device, come to the same as the launches; on fewer SMs they are right and only larger than they need to be.
//
// How a call's items are cut along their states where there are too few blocks
// of queries to go round: `parts` chunks of `chunk` states (a multiple of 128)
// each, as many as give `ctas` CTAs a block, of about `least` states at least.
struct Split {
    int parts, chunk;
};
inline Split split_of(const AttentionLaunch &L, long long blocks, long long ctas, long long least) {
    const long long most = (L.max_k + least - 1) / least;
    long long parts = blocks > 0 ? ctas / blocks : 1;
    if (parts > most) parts = most;
    if (parts > 32) parts = 32;
    if (parts < 1) parts = 1;
    return {static_cast<int>(parts), static_cast<int>(((L.max_k + parts - 1) / parts + 127) / 128 * 128)};
}
// The states of item t in part `part`.
__device__ __forceinline__ void part_of(const Split &s, int part, Item &t) {
    const int from = static_cast<int>(min(static_cast<long long>(t.nk), static_cast<long long>(part) * s.chunk));
    t.k0 += from;
    t.nk = min(s.chunk, t.nk - from);
}

// Zeroes rows of a tile: those of the first `rows` whose bit in `keep` (one
// word per 32 rows) is 0.  One warp, a row a lane; the lanes' chunks are
// staggered so that they fall into different banks.
template <int BOXES>
__device__ __forceinline__ void zero_rows(uint32_t tile, int rows, const uint32_t (&keep)[4], int lane) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const bool drop = !((keep[w] >> lane) & 1u) && 32 * w + lane < rows;
        if (!__any_sync(0xffffffffu, drop)) continue;
        if (drop)
#pragma unroll
            for (int i = 0; i < 8 * BOXES; ++i)
                st_shared_v4(tile + (i >> 3) * kBoxBytes + (32 * w + lane) * 128 + (((i + lane) & 7) << 4), 0, 0, 0, 0);
    }
}

}  // namespace attn
}  // namespace cli
