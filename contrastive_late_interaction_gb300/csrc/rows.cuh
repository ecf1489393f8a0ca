// What the kernels over whole rows share (layer norm, dropout, the residual
// join): chunks of a row, the counter-based generator behind dropout, and the
// teams of lanes or warps that take a row together.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cli_device.cuh"
#include "cli_internal.h"
#include "launch.cuh"

namespace cli {
namespace rows {

// ----------------------------------------------------------------------------
// chunks: E consecutive elements of a row, as they lie in memory
// ----------------------------------------------------------------------------

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return pack_bf16x2(a, b); }
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t *>(&h);
}

// How a call's chunks can be moved: whole (aligned to their size, and the rows
// a multiple of it), else by the widest pieces that their alignment allows,
// words of 4 bytes or halves of 2.
enum Moves { kWhole = 0, kWords = 1, kHalves = 2 };

template <typename T, int E>
struct Chunk {
    static constexpr int kBytes = E * static_cast<int>(sizeof(T)), kWords4 = kBytes / 4;
    static_assert(kBytes == 8 || kBytes == 16, "a chunk is one access");
    uint32_t w[kWords4];

    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes == 8) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(p);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kBytes == 8)
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }

    // The first n elements at p, the others 0, in words or halves.
    template <int MOVES>
    __device__ __forceinline__ void load_some(const T *p, int n) {
        if constexpr (sizeof(T) == 2 && MOVES == kHalves) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const uint32_t lo = i < n ? reinterpret_cast<const uint16_t *>(p)[i] : 0u;
                const uint32_t hi = i + 1 < n ? reinterpret_cast<const uint16_t *>(p)[i + 1] : 0u;
                w[i / 2] = lo | hi << 16;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords4; ++i) w[i] = i * E < n * kWords4 ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
        }
    }
    template <int MOVES>
    __device__ __forceinline__ void store_some(T *p, int n) const {
        if constexpr (sizeof(T) == 2 && MOVES == kHalves) {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (i < n) reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        } else {
#pragma unroll
            for (int i = 0; i < kWords4; ++i)
                if (i * E < n * kWords4) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        }
    }

    __device__ __forceinline__ void floats(float2 (&v)[E / 2]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) v[i] = unpack2<T>(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float2 (&v)[E / 2]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[2 * i] = __float_as_uint(v[i].x), w[2 * i + 1] = __float_as_uint(v[i].y);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[i] = pack2<T>(v[i].x, v[i].y);
        }
    }
};

// The n elements of a chunk that are there, from and to global memory.
template <int MOVES, typename T, int E>
__device__ __forceinline__ void take(Chunk<T, E> &c, const T *p, int n) {
    if constexpr (MOVES == kWhole) {
        if (n > 0) c.load(p);
    } else {
        c.template load_some<MOVES>(p, n);
    }
}
template <int MOVES, typename T, int E>
__device__ __forceinline__ void put(const Chunk<T, E> &c, T *p, int n) {
    if constexpr (MOVES == kWhole) {
        if (n > 0) c.store(p);
    } else {
        c.template store_some<MOVES>(p, n);
    }
}

// E consecutive floats of a vector of `width` from `at` (a multiple of 4); the vector is aligned to 4 bytes alone.  What
// lies past it, or the vector's absence, is `otherwise`.
template <int E>
__device__ __forceinline__ void vector_of(const float *p, int at, int width, float otherwise, float2 (&v)[E / 2]) {
    if (p && at + E <= width && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + at + i));
            v[i / 2] = make_float2(f.x, f.y), v[i / 2 + 1] = make_float2(f.z, f.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 2)
            v[i / 2] = make_float2(p && at + i < width ? __ldg(p + at + i) : otherwise,
                                   p && at + i + 1 < width ? __ldg(p + at + i + 1) : otherwise);
    }
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}

// A thread's chunks of one matrix, N a step, on their way to it through its own
// places in shared memory.  No other thread reads those, so that the thread's
// own wait for its copies is all that a step needs.  Halves, which no
// asynchronous copy takes, wait in registers for one step.
template <typename T, int E, int N, int MOVES>
struct Feed {
    static constexpr int kUnit = Chunk<T, E>::kBytes;
    static constexpr bool kHeld = MOVES == kHalves && sizeof(T) == 2;
    uint32_t at;   // of chunk 0 of stage 0
    Chunk<T, E> held[kHeld ? N : 1];

    // `base`: where the block's places for this matrix start, [stages][N][threads] units.  Places that no copy writes,
    // those past a row's end, are 0.
    __device__ __forceinline__ Feed(uint32_t base, int stages) {
        at = base + threadIdx.x * kUnit;
        for (int i = 0; i < stages * N; ++i) {
            if constexpr (kUnit == 16)
                st_shared_v4(at + i * blockDim.x * kUnit, 0, 0, 0, 0);
            else
                asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(at + i * blockDim.x * kUnit), "r"(0) : "memory");
        }
    }
    __device__ __forceinline__ uint32_t place(int stage, int i) const { return at + (stage * N + i) * blockDim.x * kUnit; }
    __device__ __forceinline__ void copy(int stage, int i, const T *p, int n) {
        const uint32_t to = place(stage, i);
        if constexpr (kHeld) {
            held[i].template load_some<MOVES>(p, n);
        } else if constexpr (MOVES == kWhole) {
            if (n > 0) copy_async<kUnit>(to, p);
        } else {
            constexpr int kWords4 = kUnit / 4;
#pragma unroll
            for (int k = 0; k < kWords4; ++k)
                if (k * E < n * kWords4) copy_async<4>(to + 4 * k, reinterpret_cast<const uint32_t *>(p) + k);
        }
    }
    // What is held, to its stage.
    __device__ __forceinline__ void settle(int stage) {
        if constexpr (kHeld) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(place(stage, i)), "r"(held[i].w[0]), "r"(held[i].w[1]) : "memory");
        }
    }
    __device__ __forceinline__ Chunk<T, E> chunk(int stage, int i) const {
        Chunk<T, E> c;
        if constexpr (kUnit == 16)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(c.w[0]), "=r"(c.w[1]), "=r"(c.w[2]), "=r"(c.w[3]) : "r"(place(stage, i)) : "memory");
        else
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(c.w[0]), "=r"(c.w[1]) : "r"(place(stage, i)) : "memory");
        return c;
    }
    __device__ __forceinline__ void floats(int stage, int i, float2 (&v)[E / 2]) const { chunk(stage, i).floats(v); }
};

// ----------------------------------------------------------------------------
// dropout
// ----------------------------------------------------------------------------

// Philox 4x32 of ten rounds (Salmon, Moraes, Dror, Shaw: Parallel random
// numbers: as easy as 1, 2, 3; 2011): four words of 32 bits from a counter of
// four and a key of two.
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p = static_cast<uint64_t>(0xD2511F53u) * c.x, q = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
        c = make_uint4(static_cast<uint32_t>(q >> 32) ^ c.y ^ (k0 + i * 0x9E3779B9u), static_cast<uint32_t>(q),
                       static_cast<uint32_t>(p >> 32) ^ c.w ^ (k1 + i * 0xBB67AE85u), static_cast<uint32_t>(p));
    }
    return c;
}

// A call's mask, its seed and step read from the device: a captured call draws another mask at each step.
struct Mask {
    uint32_t k0, k1, step0, step1, site, least;
    float scale;
    __device__ __forceinline__ explicit Mask(const MaskLaunch &m)
        : k0(0), k1(0), step0(0), step1(0), site(m.site << 16), least(m.least), scale(m.scale) {
        if (least) {
            const uint2 key = *reinterpret_cast<const uint2 *>(m.seed), step = *reinterpret_cast<const uint2 *>(m.seed + 1);
            // through a shuffle, which tells the compiler that these are the warp's: the rounds' keys are then added up
            // beside the other arithmetic
            k0 = __shfl_sync(0xffffffffu, key.x, 0), k1 = __shfl_sync(0xffffffffu, key.y, 0);
            step0 = __shfl_sync(0xffffffffu, step.x, 0), step1 = __shfl_sync(0xffffffffu, step.y, 0);
        }
    }
    // E elements of row `row` from column `at` (a multiple of 4): kept ones times scale, the others 0 whatever they hold.
    template <int E>
    __device__ __forceinline__ void apply(float2 (&v)[E / 2], uint32_t row, int at) const {
        if (!least) return;
#pragma unroll
        for (int i = 0; i < E / 2; i += 2) {
            const uint4 r = philox(make_uint4(static_cast<uint32_t>((at + 2 * i) >> 2) | site, row, step0, step1), k0, k1);
            v[i].x = r.x >= least ? v[i].x * scale : 0.0f;
            v[i].y = r.y >= least ? v[i].y * scale : 0.0f;
            v[i + 1].x = r.z >= least ? v[i + 1].x * scale : 0.0f;
            v[i + 1].y = r.w >= least ? v[i + 1].y * scale : 0.0f;
        }
    }
};

// ----------------------------------------------------------------------------
// teams
// ----------------------------------------------------------------------------

// Sums over a warp of N values (1, 2 or 4), the same in each lane: with several, halves of the warp take some of them each
// and hand them round at the end, 9 shuffles for four sums instead of 20.
template <int N>
__device__ __forceinline__ void warp_sum(float (&v)[N]) {
    const uint32_t lane = threadIdx.x;
    auto swap = [](float x, int o) { return __shfl_xor_sync(0xffffffffu, x, o); };
    if constexpr (N == 1) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v[0] += swap(v[0], o);
    } else if constexpr (N == 2) {
        const bool upper = lane & 16;
        float t = (upper ? v[1] : v[0]) + swap(upper ? v[0] : v[1], 16);
#pragma unroll
        for (int o = 8; o; o >>= 1) t += swap(t, o);
        const float u = swap(t, 16);
        v[0] = upper ? u : t, v[1] = upper ? t : u;
    } else {
        static_assert(N == 4, "");
        const bool upper = lane & 16, odd = lane & 8;
        const float a = (upper ? v[2] : v[0]) + swap(upper ? v[0] : v[2], 16);
        const float b = (upper ? v[3] : v[1]) + swap(upper ? v[1] : v[3], 16);
        float t = (odd ? b : a) + swap(odd ? a : b, 8);
#pragma unroll
        for (int o = 4; o; o >>= 1) t += swap(t, o);
        const float u = swap(t, 8), lo = odd ? u : t, hi = odd ? t : u, lo2 = swap(lo, 16), hi2 = swap(hi, 16);
        v[0] = upper ? lo2 : lo, v[1] = upper ? hi2 : hi, v[2] = upper ? lo : lo2, v[3] = upper ? hi : hi2;
    }
}

// The lanes that take a row together: 2^k lanes of a warp, or whole warps.
struct Team {
    int lane, lanes;      // this thread's place, the team's size
    int index, count;     // the team's place among the grid's
    int first;            // the index of the warp's first team
    int id, in_block;     // its place in the block, the block's teams
    __device__ __forceinline__ explicit Team(int lanes_) : lanes(lanes_) {
        id = threadIdx.x / lanes;
        lane = threadIdx.x - id * lanes;
        in_block = blockDim.x / lanes;
        index = blockIdx.x * in_block + id;
        count = gridDim.x * in_block;
        first = lanes < 32 ? index - (threadIdx.x & 31) / lanes : index;
    }
    // Sums of N values over the team, the same in each lane, in a fixed order.  `scratch`: 16 * N floats of the team's own
    // in shared memory, 16-byte aligned, of two that calls alternate between (a team of several warps needs one barrier a
    // sum, then).  WARPS: the team is one warp or more.
    template <int N, bool WARPS>
    __device__ __forceinline__ void sum(float (&v)[N], float *scratch) const {
        if constexpr (!WARPS) {
            for (int o = 1; o < lanes; o <<= 1) {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            }
        } else {
            warp_sum(v);
            if (lanes > 32) {
                const int warps = lanes >> 5;
                if ((lane & 31) == 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i) scratch[(lane >> 5) * N + i] = v[i];
                }
                named_barrier_sync(1 + id, lanes);
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = scratch[i];
#pragma unroll 1
                for (int w = 1; w < warps; ++w) {
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] += scratch[w * N + i];
                }
            }
        }
    }
};

}  // namespace rows
}  // namespace cli
