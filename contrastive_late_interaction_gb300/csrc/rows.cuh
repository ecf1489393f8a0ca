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

template <typename T, int E>
struct Chunk {
    static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }

    // All E elements at p, which is aligned to E elements (32 bytes are taken as two halves).
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 u = reinterpret_cast<const uint4 *>(p)[i / 4];
                w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kWords == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4)
                reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        }
    }

    // The first n elements at p, which is aligned to one; the others are 0.
    __device__ __forceinline__ void load_some(const T *p, int n) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t *>(p)[i] : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const uint32_t lo = i < n ? reinterpret_cast<const uint16_t *>(p)[i] : 0u;
                const uint32_t hi = i + 1 < n ? reinterpret_cast<const uint16_t *>(p)[i + 1] : 0u;
                w[i / 2] = lo | hi << 16;
            }
        }
    }
    __device__ __forceinline__ void store_some(T *p, int n) const {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i >= n) continue;
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(p)[i] = w[i];
            else
                reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
        }
    }

    __device__ __forceinline__ void floats(float (&v)[E]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const float2 f = unpack2<T>(w[i / 2]);
                v[i] = f.x, v[i + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void set(const float (&v)[E]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; i += 2) w[i / 2] = pack2<T>(v[i], v[i + 1]);
        }
    }
};

// A chunk's elements, of which there are n, moved as the call's alignment
// allows: E = 8 takes calls whose every matrix has rows of whole, aligned
// chunks, E = 4 the others, whole and aligned or element by element.
template <typename T, int E>
__device__ __forceinline__ void take(Chunk<T, E> &c, const T *p, int n, bool whole) {
    if (E == 8 || whole) {
        if (n > 0) c.load(p); else c.clear();
    } else {
        c.load_some(p, n);
    }
}
template <typename T, int E>
__device__ __forceinline__ void put(const Chunk<T, E> &c, T *p, int n, bool whole) {
    if (E == 8 || whole) {
        if (n > 0) c.store(p);
    } else {
        c.store_some(p, n);
    }
}

// E consecutive floats of a vector of `width`, aligned to 4 bytes alone; what lies past it, or the vector's absence, is
// `otherwise`.
template <int E>
__device__ __forceinline__ void vector_of(const float *p, int at, int width, float otherwise, float (&v)[E]) {
    if (p && at + E <= width && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {   // at is a multiple of 4
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p + at + i));
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = p && at + i < width ? __ldg(p + at + i) : otherwise;
    }
}

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
            k0 = key.x, k1 = key.y, step0 = step.x, step1 = step.y;
        }
    }
    // E elements of row `row` from column `at` (a multiple of 4): kept ones times scale, the others 0 whatever they hold.
    template <int E>
    __device__ __forceinline__ void apply(float (&v)[E], uint32_t row, int at) const {
        if (!least) return;
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const uint4 r = philox(make_uint4(static_cast<uint32_t>((at + i) >> 2) | site, row, step0, step1), k0, k1);
            v[i] = r.x >= least ? v[i] * scale : 0.0f;
            v[i + 1] = r.y >= least ? v[i + 1] * scale : 0.0f;
            v[i + 2] = r.z >= least ? v[i + 2] * scale : 0.0f;
            v[i + 3] = r.w >= least ? v[i + 3] * scale : 0.0f;
        }
    }
};

// ----------------------------------------------------------------------------
// teams
// ----------------------------------------------------------------------------

// The lanes that take a row together: 2^k lanes of a warp, or whole warps.
struct Team {
    int lane, lanes;      // this thread's place, the team's size
    int index, count;     // the team's place among the grid's
    int id, in_block;     // its place in the block, the block's teams
    __device__ __forceinline__ explicit Team(int lanes_) : lanes(lanes_) {
        id = threadIdx.x / lanes;
        lane = threadIdx.x - id * lanes;
        in_block = blockDim.x / lanes;
        index = blockIdx.x * in_block + id;
        count = gridDim.x * in_block;
    }
    // Sums of N values over the team, the same in each lane, in a fixed order.  `scratch`: N * 32 floats of the team's own
    // in shared memory, of two that calls alternate between (a team of several warps needs one barrier a sum, then).
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], float *scratch) const {
        const int within = lanes < 32 ? lanes : 32;
        for (int o = 1; o < within; o <<= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
        if (lanes > 32) {
            const int warps = lanes >> 5;
            if ((lane & 31) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) scratch[i * 32 + (lane >> 5)] = v[i];
            }
            named_barrier_sync(1 + id, lanes);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float t = 0.0f;
                for (int w = 0; w < warps; ++w) t += scratch[i * 32 + w];
                v[i] = t;
            }
        }
    }
};

}  // namespace rows
}  // namespace cli
